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
//
// 256 rows x 151936 with histories of up to 8192 tokens, masks and biases take
// 76 us, 4.2 TB/s; without histories 60, the bare copy 47. The history's
// loads, its atomics and the penalties are about 5 us each: a CTA spends them
// one after the other, and only the six on an SM cover one another. Every slice
// of a row counts its whole history: that is why slices are not shorter, and
// longer ones leave fewer CTAs. Entries per slice and time: 2048 106, 4096 85,
// 8192 76, 16384 78, 24576 88, 49152 98 us. Slower too: copies to shared memory
// ahead (95, fewer CTAs), prefetches to L2 (75 for 73).
#include <climits>

#include "common.cuh"
#include "tp_internal.h"

namespace tpk {

// V < 2^31 and a row's slice starts at most 3 entries before a multiple of
// SLICE, so that a group of four logits is 16-byte aligned in memory: group
// position 0 of slice s is vocabulary entry s * SLICE - shift, shift = (t * V)
// mod 4 entries. The groups are taken AHEAD per thread at a time, the first
// before the history is read.
template <int SLICE, int THREADS>
__global__ void __launch_bounds__(THREADS, 1536 / THREADS) logits_process_kernel(const LogitArgs a) {
    constexpr int PER = SLICE / 4 / THREADS;                // groups of four per thread
    constexpr int AHEAD = PER < 2 ? PER : 2;
    static_assert(PER % AHEAD == 0 && SLICE % (4 * THREADS) == 0, "a slice is whole rounds of every thread");
    extern __shared__ __align__(16) unsigned cnt[];         // [SLICE], a word per lane, the ids of a short bias list
    int* s_ids = reinterpret_cast<int*>(cnt + SLICE + 32);
    const int tid = threadIdx.x;
    const int t = blockIdx.x / a.slices, slice = blockIdx.x - t * a.slices;
    const int64_t row0 = (int64_t)t * a.V;
    const int shift = a.vec ? (int)(row0 & 3) : 0;
    const int v0 = slice * SLICE - shift;
    const bool in_place = a.x == a.y;
    pdl_wait();

    float4 x[AHEAD];
    auto load = [&](int v, float4& r) {
        const float* p = a.x + row0 + v;
        if (a.vec && v >= 0 && v + 3 < a.V) {
            r = __ldcs(reinterpret_cast<const float4*>(p));
        } else {
            r.x = v >= 0 && v < a.V ? p[0] : 0.f;
            r.y = v + 1 >= 0 && v + 1 < a.V ? p[1] : 0.f;
            r.z = v + 2 >= 0 && v + 2 < a.V ? p[2] : 0.f;
            r.w = v + 3 >= 0 && v + 3 < a.V ? p[3] : 0.f;
        }
    };
    auto group = [&](int i) { return v0 + 4 * (tid + i * THREADS); };
    if (!in_place && a.vec && v0 >= 0 && v0 + SLICE <= a.V)
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) load(group(i), x[i]);

    int h0 = 0, hn = 0, b0 = 0, bn = 0, np = 0;
    // entries begin .. end - 1 of a list of n: how many, 0 where they do not lie in it (negative numbers are large ones here)
    auto within = [](unsigned begin, unsigned end, unsigned n) { return begin <= end && end <= n ? (int)(end - begin) : 0; };
    float rep = 1.f, pres = 0.f, freq = 0.f;
    if (a.tokens) {
        h0 = a.cu_tokens[t];
        hn = within(h0, a.cu_tokens[t + 1], a.n_tokens);
        np = a.n_prompt ? a.n_prompt[t] : 0;
        if (a.repetition) rep = a.repetition[t];
        if (a.presence) pres = a.presence[t];
        if (a.frequency) freq = a.frequency[t];
        if (rep == 1.f && pres == 0.f && freq == 0.f) hn = 0;
    }
    if (a.bias_ids) {
        b0 = a.cu_bias[t];
        bn = within(b0, a.cu_bias[t + 1], a.n_bias);
    }
    const uint32_t* mask = nullptr;
    if (a.mask) {
        const int m = a.mask_row ? a.mask_row[t] : t;
        if (m >= 0 && m < a.mask_rows) mask = a.mask + (int64_t)m * a.mask_words;
    }
    if (in_place && !hn && !bn && !mask) return;

    const int lo = max(v0, 0), hi = (int)min((int64_t)v0 + SLICE, (int64_t)a.V);
    const unsigned span = (unsigned)max(hi - lo, 0);
    float bias = 0.f, biased = 0.f;                         // its bias and its logit, read ahead of the counting
    if (bn && bn <= THREADS && tid < bn) {
        const int id = a.bias_ids[(int64_t)b0 + tid];           // the thread's entry of a short bias list
        s_ids[tid] = id;
        if (id >= lo && id < hi) {
            bias = a.bias_values[(int64_t)b0 + tid];
            biased = a.x[row0 + id];
        }
    }
    if (hn) {
        for (int i = tid; i < SLICE / 4; i += THREADS) reinterpret_cast<uint4*>(cnt)[i] = make_uint4(0, 0, 0, 0);
        __syncthreads();
        // Every token counts somewhere, one outside the slice in a word of its lane behind it: no branch, which would
        // cost more than the count. Four tokens per load, four loads in flight.
        const int out = SLICE + (tid & 31) - lo + v0;
        auto scan = [&](const int* h, int n, auto&& count) {
            auto one = [&](int tok) {
                const unsigned u = (unsigned)tok - (unsigned)lo;
                count(&cnt[(int)(u < span ? u : (unsigned)out) + (lo - v0)]);
            };
            auto four = [&](const int4& w) {
                one(w.x);
                one(w.y);
                one(w.z);
                one(w.w);
            };
            const int head = min((int)(((16 - (reinterpret_cast<uintptr_t>(h) & 15)) >> 2) & 3), n), nv = (n - head) >> 2;
            if (tid < head) one(h[tid]);
            const int4* h4 = reinterpret_cast<const int4*>(h + head);
            int j = tid;
            for (; j + 3 * THREADS < nv; j += 4 * THREADS) {
                int4 w[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) w[k] = h4[j + k * THREADS];
#pragma unroll
                for (int k = 0; k < 4; ++k) four(w[k]);
            }
            for (; j < nv; j += THREADS) four(h4[j]);
            if (head + 4 * nv + tid < n) one(h[head + 4 * nv + tid]);
        };
        const int n0 = min(max(np, 0), hn);
        scan(a.tokens + h0, n0, [](unsigned* w) { atomicOr(w, 1u); });
        scan(a.tokens + h0 + n0, hn - n0, [](unsigned* w) { atomicAdd(w, 2u); });
        __syncthreads();
    }

    // mask bits of the entries v .. v + 3, some of which may be out of range
    auto allowed4 = [&](int v) -> unsigned {
        const int va = min(max(v, 0), a.V - 1), vb = min(max(v + 3, 0), a.V - 1);
        const uint32_t w0 = mask[va >> 5], w1 = mask[vb >> 5];
        return (v >= 0 ? __funnelshift_r(w0, w1, v & 31) : w0 << -v) & 15u;
    };
    auto penalise = [&](float e, unsigned n) {
        e = e > 0.f ? e / rep : e * rep;
        return n > 1u ? e - freq * (float)(n >> 1) - pres : e;
    };
    auto change = [&](float4& x, const uint4& c, unsigned ok) {
        float e[4] = {x.x, x.y, x.z, x.w};
        const unsigned n[4] = {c.x, c.y, c.z, c.w};
        // one at a time: most groups have none, but most warps have one in a lane, and four of them in turn would cost
        // the warp four divisions
        unsigned any = (n[0] ? 1u : 0u) | (n[1] ? 2u : 0u) | (n[2] ? 4u : 0u) | (n[3] ? 8u : 0u);
#pragma unroll 1
        for (; any; any &= any - 1) {
            const unsigned k = any & -any;
            const float z = penalise(k == 1 ? e[0] : k == 2 ? e[1] : k == 4 ? e[2] : e[3],
                                     k == 1 ? n[0] : k == 2 ? n[1] : k == 4 ? n[2] : n[3]);
            e[0] = k == 1 ? z : e[0];
            e[1] = k == 2 ? z : e[1];
            e[2] = k == 4 ? z : e[2];
            e[3] = k == 8 ? z : e[3];
        }
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (!(ok >> k & 1u)) e[k] = -INFINITY;
        x = make_float4(e[0], e[1], e[2], e[3]);
    };
    if (!in_place && a.vec && v0 >= 0 && v0 + SLICE <= a.V) {
        // A slice inside its row, the common case: every address is the thread's first and a constant, and the thread's
        // groups have their mask bits at the same place of words a constant apart.
        const int first = group(0), sh = first & 31;
        const float4* px = reinterpret_cast<const float4*>(a.x + row0 + first);
        float4* py = reinterpret_cast<float4*>(a.y + row0 + first);
        const uint32_t* pm = mask ? mask + (first >> 5) : nullptr;
        const uint4* pc = reinterpret_cast<const uint4*>(cnt) + tid;
#pragma unroll
        for (int c = 0; c < PER; c += AHEAD) {
            if (c)
#pragma unroll
                for (int i = 0; i < AHEAD; ++i) x[i] = __ldcs(px + (c + i) * THREADS);
            unsigned ok[AHEAD];
#pragma unroll
            for (int i = 0; i < AHEAD; ++i) {
                ok[i] = 15u;
                if (mask) {
                    const uint32_t* w = pm + (c + i) * (THREADS / 8);
                    ok[i] = __funnelshift_r(w[0], sh > 28 ? w[1] : 0u, sh);
                }
            }
#pragma unroll
            for (int i = 0; i < AHEAD; ++i) {
                change(x[i], hn ? pc[(c + i) * THREADS] : make_uint4(0, 0, 0, 0), ok[i]);
                __stcs(py + (c + i) * THREADS, x[i]);
            }
        }
    } else {
#pragma unroll 1
        for (int i = 0; i < PER; ++i) {
            const int v = group(i);
            if (v >= a.V || v + 3 < 0) continue;
            const uint4 c = hn ? reinterpret_cast<const uint4*>(cnt)[tid + i * THREADS] : make_uint4(0, 0, 0, 0);
            const unsigned ok = mask ? allowed4(v) : 15u;
            if (in_place && !(c.x | c.y | c.z | c.w) && ok == 15u) continue;
            float4 z;
            load(v, z);
            change(z, c, ok);
            float* p = a.y + row0 + v;
            if (a.vec && v >= 0 && v + 3 < a.V) {
                *reinterpret_cast<float4*>(p) = z;
            } else {
                if (v >= 0) p[0] = z.x;
                if (v + 1 >= 0 && v + 1 < a.V) p[1] = z.y;
                if (v + 2 >= 0 && v + 2 < a.V) p[2] = z.z;
                if (v + 3 < a.V) p[3] = z.w;
            }
        }
    }

    // Biases go onto the penalised logits; a masked one stays -inf. The results of a short list are formed from what was read
    // ahead and replace what the sweep has written, those of a long one are added to it.
    if (!bn) return;
    __syncthreads();
    auto add = [&](int v, int entry) {
        if (!mask || mask[v >> 5] >> (v & 31) & 1u) a.y[row0 + v] += a.bias_values[(int64_t)b0 + entry];
    };
    if (bn <= THREADS) {
        const int id = tid < bn ? s_ids[tid] : -1;
        if (id >= lo && id < hi) {
            bool last = true;
            for (int j = tid + 1; j < bn; ++j) last &= s_ids[j] != id;
            const unsigned n = hn ? cnt[id - v0] : 0u;
            if (n) biased = penalise(biased, n);
            if (last && (!mask || mask[id >> 5] >> (id & 31) & 1u)) a.y[row0 + id] = biased + bias;
        }
        return;
    }
    for (int i = tid; i < SLICE / 4; i += THREADS) reinterpret_cast<uint4*>(cnt)[i] = make_uint4(0, 0, 0, 0);
    __syncthreads();
    for (int i = tid; i < bn; i += THREADS) {
        const int tok = a.bias_ids[(int64_t)b0 + i];
        if (tok >= lo && tok < hi) atomicMax(&cnt[tok - v0], (unsigned)i + 1u);
    }
    __syncthreads();
    for (int u = tid; u < SLICE; u += THREADS)
        if (cnt[u]) add(v0 + u, (int)cnt[u] - 1);
}

template <int SLICE, int THREADS>
static cudaError_t launch_slices(LogitArgs a, cudaStream_t s) {
    a.slices = (int)(((int64_t)a.V + 3 + SLICE - 1) / SLICE);
    const int64_t grid = (int64_t)a.T * a.slices;
    if (grid > INT_MAX) return cudaErrorInvalidConfiguration;
    constexpr size_t smem = (SLICE + 32 + THREADS) * sizeof(unsigned);
    static_assert(smem <= 48 * 1024, "what a kernel gets without asking");
    void* args[] = {&a};
    return launch_pdl(reinterpret_cast<const void*>(logits_process_kernel<SLICE, THREADS>), args, (int)grid, smem, s, THREADS);
}

cudaError_t launch_logits(const LogitArgs& a, cudaStream_t s) {
    return launch_slices<8192, 256>(a, s);
}

}  // namespace tpk
