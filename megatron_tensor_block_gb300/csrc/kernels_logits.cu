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
// 1..: generated occurrences); integer atomics, so their order does not change
// a result. One sweep then reads, changes and writes each logit once; its
// logits are loaded into registers before the history is counted. The few
// biased entries follow.
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
    __shared__ __align__(16) unsigned cnt[SLICE];
    __shared__ int s_ids[kLogitThreads];
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

    const int lo = max(v0, 0), hi = (int)min((int64_t)v0 + SLICE, (int64_t)a.V);
    int id = -1;                                            // the thread's entry of a short bias list
    if (bn && bn <= kLogitThreads && tid < bn) s_ids[tid] = id = a.bias_ids[(int64_t)b0 + tid];
    if (hn) {
        for (int i = tid; i < SLICE / 4; i += kLogitThreads) reinterpret_cast<uint4*>(cnt)[i] = make_uint4(0, 0, 0, 0);
        __syncthreads();
        auto hit = [&](int tok, int i) {
            if (tok < lo || tok >= hi) return;
            if (i < np) atomicOr(&cnt[tok - v0], 1u);
            else atomicAdd(&cnt[tok - v0], 2u);
        };
        // four tokens per load, four loads in flight
        const int* h = a.tokens + h0;
        const int head = min((int)(((16 - (reinterpret_cast<uintptr_t>(h) & 15)) >> 2) & 3), hn), nv = (hn - head) >> 2;
        if (tid < head) hit(h[tid], tid);
        const int4* h4 = reinterpret_cast<const int4*>(h + head);
        for (int j = tid; j < nv; j += 4 * kLogitThreads) {
            int4 w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) w[k] = j + k * kLogitThreads < nv ? h4[j + k * kLogitThreads] : make_int4(-1, -1, -1, -1);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int i = head + 4 * (j + k * kLogitThreads);
                hit(w[k].x, i);
                hit(w[k].y, i + 1);
                hit(w[k].z, i + 2);
                hit(w[k].w, i + 3);
            }
        }
        for (int i = head + 4 * nv + tid; i < hn; i += kLogitThreads) hit(h[i], i);
        __syncthreads();
    }
    auto allowed4 = [&](int v) -> unsigned {                // mask bits of entries v .. v + 3
        if (!mask) return 15u;
        const int va = max(v, 0), vb = min(v + 3, a.V - 1);
        const uint32_t w0 = mask[va >> 5], w1 = mask[vb >> 5];
        return (v >= 0 ? __funnelshift_r(w0, w1, v & 31) : w0 << -v) & 15u;
    };

#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int g = tid + i * kLogitThreads, v = v0 + 4 * g;
        if (v >= a.V || v + 3 < 0) continue;
        const uint4 c4 = hn ? reinterpret_cast<const uint4*>(cnt)[g] : make_uint4(0, 0, 0, 0);
        const unsigned allowed = allowed4(v);
        const bool touched = (c4.x | c4.y | c4.z | c4.w) || allowed != 15u;
        if (in_place) {
            if (!touched) continue;
            load(v, x[i]);
        }
        float e[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
        if (touched) {
            const unsigned c[4] = {c4.x, c4.y, c4.z, c4.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if (c[k]) {
                    e[k] = e[k] > 0.f ? e[k] / rep : e[k] * rep;
                    if (c[k] > 1u) e[k] = e[k] - freq * (float)(c[k] >> 1) - pres;
                }
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

    // Biases go onto the penalised logits that the sweep has written; a masked one stays -inf.
    if (!bn) return;
    __syncthreads();
    auto add = [&](int v, int entry) {
        if (allowed4(v) & 1u) a.y[row0 + v] += a.bias_values[(int64_t)b0 + entry];
    };
    if (bn <= kLogitThreads) {
        if (id >= lo && id < hi) {
            bool last = true;
            for (int j = tid + 1; j < bn; ++j) last &= s_ids[j] != id;
            if (last) add(id, tid);
        }
        return;
    }
    for (int i = tid; i < SLICE / 4; i += kLogitThreads) reinterpret_cast<uint4*>(cnt)[i] = make_uint4(0, 0, 0, 0);
    __syncthreads();
    for (int i = tid; i < bn; i += kLogitThreads) {
        const int tok = a.bias_ids[(int64_t)b0 + i];
        if (tok >= lo && tok < hi) atomicMax(&cnt[tok - v0], (unsigned)i + 1u);
    }
    __syncthreads();
    for (int u = tid; u < SLICE; u += kLogitThreads)
        if (cnt[u]) add(v0 + u, (int)cnt[u] - 1);
}

template <int SLICE>
static cudaError_t launch_slices(LogitArgs a, cudaStream_t s) {
    a.slices = (int)(((int64_t)a.V + 3 + SLICE - 1) / SLICE);
    const int64_t grid = (int64_t)a.T * a.slices;
    if (grid > INT_MAX) return cudaErrorInvalidConfiguration;
    void* args[] = {&a};
    return launch_pdl(reinterpret_cast<const void*>(logits_process_kernel<SLICE>), args, (int)grid, 0, s, kLogitThreads);
}

cudaError_t launch_logits(const LogitArgs& a, cudaStream_t s) {
    return launch_slices<8192>(a, s);
}

}  // namespace tpk
