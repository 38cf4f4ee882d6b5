// Per-row controls of a batch's logits: penalties for tokens of the row's
// history, biases, grammar masks.
//
//   y = x > 0 ? x / r : x * r  for tokens of the history, then
//   y -= f * c + a             for tokens with c > 0 generated occurrences, then
//   y += bias, then y = -inf   where the row's mask bit is 0.
//
// The pass is bound by memory: 4 bytes in and 4 out per logit (in place: only
// what a control changes), plus an eighth of a byte of mask. A CTA takes one
// slice of one row's vocabulary. It counts the row's whole history into one
// shared-memory word per token of its slice (bit 0: seen in the prompt, bits
// 1..: generated occurrences) and the last bias entry per token into another;
// integer atomics, so their order does not change a result. One sweep then
// reads, changes and writes each logit once. The logits of the sweep are
// loaded into registers before the history is counted.
#include <climits>

#include "common.cuh"
#include "tp_internal.h"

namespace tpk {

constexpr int kLogitThreads = 256;

// V < 2^31 and a row's slice starts at most 3 entries before a multiple of
// SLICE, so that a group of four logits is 16-byte aligned in memory: group
// position 0 of slice s is vocabulary entry s * SLICE - shift, shift = (t * V)
// mod 4 entries.
template <int SLICE>
__global__ void __launch_bounds__(kLogitThreads) logits_process_kernel(const LogitArgs a) {
    constexpr int PER = SLICE / 4 / kLogitThreads;          // groups of four per thread
    static_assert(PER >= 1 && SLICE % (4 * kLogitThreads) == 0, "a slice is whole groups of every thread");
    extern __shared__ __align__(16) unsigned s_words[];
    unsigned* cnt = s_words;
    unsigned* last = s_words + SLICE;
    const int tid = threadIdx.x;
    const int t = blockIdx.x / a.slices, slice = blockIdx.x - t * a.slices;
    const int64_t row0 = (int64_t)t * a.V;
    const int shift = a.vec ? (int)(row0 & 3) : 0;
    const int v0 = slice * SLICE - shift;
    const bool in_place = a.x == a.y;
    pdl_wait();

    int h0 = 0, hn = 0, b0 = 0, bn = 0, np = 0;
    float rep = 1.f, pres = 0.f, freq = 0.f;
    if (a.tokens) {
        h0 = a.cu_tokens[t];
        hn = max(a.cu_tokens[t + 1] - h0, 0);
        np = a.n_prompt ? a.n_prompt[t] : 0;
        if (a.repetition) rep = a.repetition[t];
        if (a.presence) pres = a.presence[t];
        if (a.frequency) freq = a.frequency[t];
        if (rep == 1.f && pres == 0.f && freq == 0.f) hn = 0;
    }
    if (a.bias_ids) {
        b0 = a.cu_bias[t];
        bn = max(a.cu_bias[t + 1] - b0, 0);
    }
    const uint32_t* mask = nullptr;
    if (a.mask) {
        const int m = a.mask_row ? a.mask_row[t] : t;
        if (m >= 0 && m < a.mask_rows) mask = a.mask + (int64_t)m * a.mask_words;
    }
    if (in_place && !hn && !bn && !mask) return;

    // the thread's logits: groups tid, tid + 256, ... of the slice
    float4 x[PER];
    const bool ahead = !in_place;
    auto load = [&](int v, float4& r) {
        const float* p = a.x + row0 + v;
        if (a.vec && v >= 0 && v + 3 < a.V) {
            r = *reinterpret_cast<const float4*>(p);
        } else {
            r.x = v >= 0 && v < a.V ? p[0] : 0.f;
            r.y = v + 1 >= 0 && v + 1 < a.V ? p[1] : 0.f;
            r.z = v + 2 >= 0 && v + 2 < a.V ? p[2] : 0.f;
            r.w = v + 3 >= 0 && v + 3 < a.V ? p[3] : 0.f;
        }
    };
    if (ahead)
#pragma unroll
        for (int i = 0; i < PER; ++i) load(v0 + 4 * (tid + i * kLogitThreads), x[i]);

    if (hn)
        for (int i = tid; i < SLICE / 4; i += kLogitThreads) reinterpret_cast<uint4*>(cnt)[i] = make_uint4(0, 0, 0, 0);
    if (bn)
        for (int i = tid; i < SLICE / 4; i += kLogitThreads) reinterpret_cast<uint4*>(last)[i] = make_uint4(0, 0, 0, 0);
    if (hn || bn) __syncthreads();
    const int lo = max(v0, 0), hi = min((int64_t)v0 + SLICE, (int64_t)a.V);
    for (int i = tid; i < hn; i += kLogitThreads) {
        const int tok = a.tokens[(int64_t)h0 + i];
        if (tok < lo || tok >= hi) continue;
        if (i < np) atomicOr(&cnt[tok - v0], 1u);
        else atomicAdd(&cnt[tok - v0], 2u);
    }
    for (int i = tid; i < bn; i += kLogitThreads) {
        const int tok = a.bias_ids[(int64_t)b0 + i];
        if (tok >= lo && tok < hi) atomicMax(&last[tok - v0], (unsigned)i + 1u);
    }
    if (hn || bn) __syncthreads();

#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int g = tid + i * kLogitThreads, v = v0 + 4 * g;
        if (v >= a.V || v + 3 < 0) continue;
        const uint4 c4 = hn ? reinterpret_cast<const uint4*>(cnt)[g] : make_uint4(0, 0, 0, 0);
        const uint4 l4 = bn ? reinterpret_cast<const uint4*>(last)[g] : make_uint4(0, 0, 0, 0);
        unsigned allowed = 15u;
        if (mask) {
            const int va = max(v, 0), vb = min(v + 3, a.V - 1);
            const uint32_t w0 = mask[va >> 5], w1 = mask[vb >> 5];
            allowed = (v >= 0 ? __funnelshift_r(w0, w1, v & 31) : w0 << -v) & 15u;
        }
        const bool touched = (c4.x | c4.y | c4.z | c4.w | l4.x | l4.y | l4.z | l4.w) || allowed != 15u;
        if (in_place) {
            if (!touched) continue;
            load(v, x[i]);
        }
        float e[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
        if (touched) {
            const unsigned c[4] = {c4.x, c4.y, c4.z, c4.w}, l[4] = {l4.x, l4.y, l4.z, l4.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if (c[k]) {
                    e[k] = e[k] > 0.f ? e[k] / rep : e[k] * rep;
                    if (c[k] > 1u) e[k] = e[k] - freq * (float)(c[k] >> 1) - pres;
                }
                if (l[k]) e[k] += a.bias_values[(int64_t)b0 + l[k] - 1];
                if (!((allowed >> k) & 1u)) e[k] = -INFINITY;
            }
        }
        float* p = a.y + row0 + v;
        if (a.vec && v >= 0 && v + 3 < a.V) {
            *reinterpret_cast<float4*>(p) = make_float4(e[0], e[1], e[2], e[3]);
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (v + k >= 0 && v + k < a.V) p[k] = e[k];
        }
    }
}

template <int SLICE>
static cudaError_t launch_slices(LogitArgs a, cudaStream_t s) {
    a.slices = (int)(((int64_t)a.V + 3 + SLICE - 1) / SLICE);
    const int64_t grid = (int64_t)a.T * a.slices;
    if (grid > INT_MAX) return cudaErrorInvalidConfiguration;
    const size_t smem = (a.bias_ids ? 2 : 1) * SLICE * sizeof(unsigned);
    const void* fn = reinterpret_cast<const void*>(logits_process_kernel<SLICE>);
    if (smem > 48 * 1024) {
        cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
    }
    void* args[] = {&a};
    return launch_pdl(fn, args, (int)grid, smem, s, kLogitThreads);
}

cudaError_t launch_logits(const LogitArgs& a, cudaStream_t s) {
    return launch_slices<8192>(a, s);
}

}  // namespace tpk
