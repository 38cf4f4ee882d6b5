// Attention of a packed batch over 8-bit pages.
//
//   o = sum_j w_j v_j / sum_j w_j,  w_j = 2^(s_j - m),  s_j = q . k_j log2(e) / sqrt(d)
//
// A warp per query row and head walks the keys, 32 at a time: a lane has a key
// for the scores and d / 32 features for the sums.
#include "common.cuh"
#include "tp_internal.h"

namespace tpk {

__device__ __forceinline__ float from_e4m3(uint8_t x) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)x));
    float f;
    asm("{\n\t.reg .f16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.f32.f16 %0, l;\n\t}" : "=f"(f) : "r"(h));
    return f;
}

template <int D>
__global__ void __launch_bounds__(128) paged_rows_kernel(const __grid_constant__ PagedAttnArgs p) {
    __shared__ float sq[4][D];
    int bad = 0;
    for (int i = threadIdx.x; i < p.B; i += blockDim.x) {
        const int a = p.cu[i], b = p.cu[i + 1];
        bad |= b < a || a < 0 || b > p.T || (i == 0 && a != 0);
    }
    if (__syncthreads_or(bad)) {
        if (threadIdx.x == 0 && blockIdx.x == 0) set_status(p.status, TP_ERR_SHAPE);
        return;
    }
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t unit = (int64_t)blockIdx.x * 4 + warp, heads = (int64_t)p.N * p.hq_s;
    const int t = (int)(unit / heads), hh = (int)(unit - t * heads), r = hh / p.hq_s, h = hh - r * p.hq_s;
    if (t >= p.cu[p.B]) return;
    int b = 0;
    for (int lo = 0, hi = p.B; hi - lo > 1;) {
        const int m = (lo + hi) >> 1;
        if (p.cu[m] <= t) lo = b = m;
        else hi = m;
    }
    if (p.cu[b + 1] - p.cu[b] > p.max_new) {
        if (lane == 0) set_status(p.status, TP_ERR_SHAPE);
        return;
    }
    const int64_t pos = (int64_t)p.pos[b] + (t - p.cu[b]), cap = (int64_t)p.c.width * p.c.page;
    bf16* out = static_cast<bf16*>(p.out) + (((int64_t)r * p.T + t) * p.hq_s + h) * D;
    if (pos < 0 || pos >= cap) {
        if (lane == 0) set_status(p.status, TP_ERR_CAPACITY);
        for (int i = lane; i < D; i += 32) out[i] = __float2bfloat16_rn(0.f);
        return;
    }
    const bf16* q = static_cast<const bf16*>(p.q) + (((int64_t)r * p.T + t) * p.hq_s + h) * D;
    for (int i = lane; i < D; i += 32) sq[warp][i] = __bfloat162float(q[i]) * p.scale_log2;
    __syncwarp();
    const int kv = h / (p.hq_s / p.hkv_s), bits = 31 - __clz(p.c.page);
    float m = -INFINITY, l = 0.f, o[D / 32] = {};
    bool any = false;
    for (int64_t j0 = 0; j0 <= pos; j0 += 32) {
        const int64_t j = j0 + lane;
        const int id = j <= pos ? p.c.pages[(int64_t)b * p.c.width + (j >> bits)] : -1;
        const bool seen = id >= 0 && id < p.c.n_pages;
        if (j <= pos && !seen) set_status(p.status, TP_ERR_CAPACITY);
        const int64_t tile = (int64_t)id * p.hkv_s + kv;
        float s = -INFINITY;
        if (seen) {
            const uint8_t* k = p.c.k[r] + (tile * p.c.page + (j & (p.c.page - 1))) * D;
            float x = 0.f;
            for (int i = 0; i < D; ++i) x = fmaf(sq[warp][i], from_e4m3(k[i]), x);
            s = x * p.c.ks[r][tile];
        }
        any |= __any_sync(0xffffffffu, seen);
        const float top = fmaxf(m, warp_max(s)), base = top == -INFINITY ? 0.f : top;
        const float w = seen ? ex2_approx(s - base) : 0.f, keep = m == -INFINITY ? 0.f : ex2_approx(m - base);
        m = top;
        l = l * keep + warp_sum(w);
        for (int i = 0; i < D / 32; ++i) o[i] *= keep;
        for (int i = 0; i < 32; ++i) {
            const int64_t from = __shfl_sync(0xffffffffu, tile, i);
            const float wi = __shfl_sync(0xffffffffu, w, i);
            if (!__shfl_sync(0xffffffffu, (int)seen, i)) continue;
            const uint8_t* v = p.c.v[r] + (from * p.c.page + ((j0 + i) & (p.c.page - 1))) * D;
            const float f = wi * p.c.vs[r][from];
            for (int x = 0; x < D / 32; ++x) o[x] = fmaf(f, from_e4m3(v[lane + 32 * x]), o[x]);
        }
    }
    for (int x = 0; x < D / 32; ++x) out[lane + 32 * x] = __float2bfloat16_rn(any ? o[x] / l : 0.f);
}

size_t paged_workspace(int64_t max_tokens, int group, int d) { return kPagedCtrl; }

cudaError_t launch_attn_paged(const PagedAttnArgs& p, cudaStream_t s) {
    PagedAttnArgs a = p;
    const int64_t units = (int64_t)a.T * a.N * a.hq_s;
    if (a.d == 128) paged_rows_kernel<128><<<(unsigned)((units + 3) / 4), 128, 0, s>>>(a);
    else paged_rows_kernel<64><<<(unsigned)((units + 3) / 4), 128, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace tpk
