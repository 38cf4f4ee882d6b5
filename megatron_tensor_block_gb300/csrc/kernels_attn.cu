// Attention of a packed batch over the shards' KV caches, with an optional
// prefix that the batch shares.
#include <climits>

#include "common.cuh"
#include "tp_internal.h"

namespace tpk {

// Checks the batch's offsets and positions: ctl->n_tokens = cu[B], or 0 with
// TP_ERR_SHAPE in the status word where cu is malformed; TP_ERR_CAPACITY where
// a token's position is outside the cache.
__global__ void __launch_bounds__(256) attn_check_kernel(const RaggedAttnParams p) {
    pdl_wait();
    int bad = 0, out = 0;
    for (int b = threadIdx.x; b < p.B; b += 256) {
        const int c0 = p.cu[b], c1 = p.cu[b + 1];
        if (c1 < c0 || c0 < 0 || c1 > p.T || (b == 0 && c0 != 0)) bad = 1;
        else if (c1 > c0 && (p.pos[b] < 0 || (int64_t)p.pos[b] + (c1 - c0) > p.max_kv)) out = 1;
    }
    bad = __syncthreads_or(bad);
    out = __syncthreads_or(out);
    if (threadIdx.x == 0) {
        p.ctl->n_tokens = bad ? 0 : p.cu[p.B];
        if (bad) set_status(p.status, TP_ERR_SHAPE);
        else if (out) set_status(p.status, TP_ERR_CAPACITY);
    }
}

// One warp per (shard, token, query head); a lane takes one key of 32 for the
// scores and D / 32 output elements for the sums.
template <int D>
__global__ void __launch_bounds__(256) attn_rows_kernel(const RaggedAttnParams p) {
    __shared__ float sq[8][D];
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t unit = (int64_t)blockIdx.x * 8 + w;
    const int h = (int)(unit % p.hq_s);
    const int t = (int)(unit / p.hq_s % p.T), r = (int)(unit / p.hq_s / p.T);
    pdl_wait();
    if (r >= p.N || t >= p.ctl->n_tokens) return;
    int b = 0;
    for (int lo = 0, hi = p.B - 1; lo <= hi;) {          // the last b with cu[b] <= t
        const int m = (lo + hi) >> 1;
        if (p.cu[m] <= t) b = m, lo = m + 1;
        else hi = m - 1;
    }
    const int64_t pos = (int64_t)p.pos[b] + (t - p.cu[b]);
    const bool in = pos >= 0 && pos < p.max_kv;
    const int kvh = h / (p.hq_s / p.hkv_s);
    const bf16* q = static_cast<const bf16*>(p.q) + (((int64_t)r * p.T + t) * p.hq_s + h) * D;
    for (int i = lane; i < D; i += 32) sq[w][i] = __bfloat162float(q[i]) * p.scale_log2;
    __syncwarp();
    float m = -INFINITY, l = 0.f, o[D / 32] = {};
    auto run = [&](const bf16* k, const bf16* v, int64_t n) {
        for (int64_t j0 = 0; j0 < n; j0 += 32) {
            float s = -INFINITY;
            if (j0 + lane < n) {
                s = 0.f;
                for (int i = 0; i < D; ++i) s = fmaf(sq[w][i], __bfloat162float(k[(j0 + lane) * D + i]), s);
            }
            const float mn = fmaxf(m, warp_max(s)), alpha = exp2f(m - mn), e = j0 + lane < n ? exp2f(s - mn) : 0.f;
            m = mn;
            l = l * alpha + warp_sum(e);
            for (int i = 0; i < D / 32; ++i) o[i] *= alpha;
            for (int j = 0; j < 32 && j0 + j < n; ++j) {
                const float pj = __shfl_sync(0xffffffffu, e, j);
                for (int i = 0; i < D / 32; ++i) o[i] = fmaf(pj, __bfloat162float(v[(j0 + j) * D + lane + 32 * i]), o[i]);
            }
        }
    };
    if (in) {
        if (p.prefix_len) {
            const int64_t off = (int64_t)kvh * p.prefix_rows * D;
            run(static_cast<const bf16*>(p.pk[r]) + off, static_cast<const bf16*>(p.pv[r]) + off, p.prefix_len);
        }
        const int64_t off = ((int64_t)b * p.hkv_s + kvh) * p.max_kv * D;
        run(static_cast<const bf16*>(p.kc[r]) + off, static_cast<const bf16*>(p.vc[r]) + off, pos + 1);
    }
    bf16* out = static_cast<bf16*>(p.out) + (((int64_t)r * p.T + t) * p.hq_s + h) * D;
    for (int i = 0; i < D / 32; ++i) out[lane + 32 * i] = __float2bfloat16_rn(in ? o[i] / l : 0.f);
}

cudaError_t launch_attn_check(const RaggedAttnParams& p, cudaStream_t s) {
    RaggedAttnParams a = p;
    void* args[] = {&a};
    return launch_pdl(reinterpret_cast<const void*>(attn_check_kernel), args, 1, 0, s, 256);
}

cudaError_t launch_attn_ragged(const RaggedAttnParams& p, cudaStream_t s) {
    const int64_t grid = ((int64_t)p.N * p.T * p.hq_s + 7) / 8;
    if (grid > INT_MAX) return cudaErrorInvalidConfiguration;
    const void* fn = p.d == 128 ? reinterpret_cast<const void*>(attn_rows_kernel<128>)
                                : reinterpret_cast<const void*>(attn_rows_kernel<64>);
    RaggedAttnParams a = p;
    void* args[] = {&a};
    return launch_pdl(fn, args, (int)grid, 0, s, 256);
}

}  // namespace tpk
