// Rotary embedding of a packed batch, and appending its keys and values to
// 8-bit pages with that rotation on the way.
//
// A pair (a, b) of features turns by the angle p f: the host gives f as a
// 64-bit fraction of a turn per position, and p times it modulo 2^64 is the
// angle modulo a turn, exact for that f however far p is (a float32 product
// p f is off by whole degrees at p = 10^6). The nearest quarter turn is taken
// off as an integer, so that sine and cosine are taken of at most an eighth.
#include "common.cuh"
#include "e4m3.cuh"
#include "tp_internal.h"

namespace tpk {

constexpr int kPgThreads = 256;
constexpr int kPgRows = 16;               // token rows whose sines are in shared memory at a time

// Whether cu is not 0 = cu[0] <= cu[1] <= ... <= T (the whole block asks).
__device__ __forceinline__ bool cu_malformed(const int* cu, int B, int T) {
    int bad = 0;
    for (int i = threadIdx.x; i < B; i += blockDim.x) {
        const int a = cu[i], b = cu[i + 1];
        bad |= b < a || a < 0 || b > T || (i == 0 && a != 0);
    }
    return __syncthreads_or(bad);
}

// The sequence of token row t < cu[B]: the last with cu[b] <= t.
__device__ __forceinline__ int sequence_of(const int* cu, int B, int t) {
    int lo = 0, hi = B;                   // cu[lo] <= t < cu[hi]
    while (hi - lo > 1) {
        const int m = (lo + hi) >> 1;
        if (__ldg(cu + m) <= t) lo = m;
        else hi = m;
    }
    return lo;
}

__device__ __forceinline__ float2 cos_sin(int64_t p, uint64_t turn, float by) {
    const uint64_t x = (uint64_t)p * turn, quarter = (x + (1ull << 61)) >> 62;
    float s, c;
    sincospif(__ll2float_rn((int64_t)(x - (quarter << 62))) * 0x1p-63f, &s, &c);
    if (quarter & 1) {
        const float t = c;
        c = -s;
        s = t;
    }
    if (quarter & 2) c = -c, s = -s;
    return make_float2(c * by, s * by);
}

__device__ __forceinline__ void load8(const bf16* p, float (&x)[8]) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = unpack_bf16x2(w[i]);
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
    }
}
__device__ __forceinline__ void load8(const float* p, float (&x)[8]) {
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}
__device__ __forceinline__ void store8(bf16* p, const float (&x)[8]) {
    *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                                              pack_bf16x2(x[6], x[7]));
}
__device__ __forceinline__ void store8(float* p, const float (&x)[8]) {
    reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}

// A unit is sixteen features of a head: eight pairs, or features behind the
// rotated ones. Features of its two halves.
__device__ __forceinline__ void unit_at(const RopeTable& r, int u, int& a, int& b) {
    const bool half = r.layout == TP_ROPE_HALF && 16 * u < r.rot;
    a = half ? 8 * u : 16 * u;
    b = half ? r.rot / 2 + 8 * u : 16 * u + 8;
}
// ... turned; cs: the row's cosines and sines.
__device__ __forceinline__ void turn_unit(const RopeTable& r, int u, const float2* cs, float (&a)[8], float (&b)[8]) {
    if (16 * u >= r.rot) return;
    if (r.layout == TP_ROPE_HALF) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float2 t = cs[8 * u + i];
            const float x = a[i], y = b[i];
            a[i] = x * t.x - y * t.y;
            b[i] = x * t.y + y * t.x;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
            const float2 t = cs[8 * u + i / 2], v = cs[8 * u + 4 + i / 2];
            float x = a[i], y = a[i + 1];
            a[i] = x * t.x - y * t.y;
            a[i + 1] = x * t.y + y * t.x;
            x = b[i], y = b[i + 1];
            b[i] = x * v.x - y * v.y;
            b[i + 1] = x * v.y + y * v.x;
        }
    }
}

// One CTA: `rows` token rows of a shard. Bound by the bytes of the rows.
template <typename T>
__global__ void __launch_bounds__(kPgThreads) rope_kernel(const __grid_constant__ RopeArgs p, int rows) {
    __shared__ float2 cs[kPgRows][64];
    __shared__ int64_t s_pos[kPgRows];
    const int tid = threadIdx.x;
    if (cu_malformed(p.cu, p.B, p.T)) {
        if (tid == 0 && blockIdx.x == 0) set_status(p.status, TP_ERR_SHAPE);
        return;
    }
    const int r = blockIdx.x % p.N, t0 = blockIdx.x / p.N * rows, n = min(rows, __ldg(p.cu + p.B) - t0);
    if (n <= 0) return;
    if (tid < n) {
        const int b = sequence_of(p.cu, p.B, t0 + tid);
        s_pos[tid] = (int64_t)p.pos[b] + (t0 + tid - p.cu[b]);
    }
    __syncthreads();
    const int half = p.rope.rot / 2;
    for (int i = tid; i < n * half; i += kPgThreads) {
        const int t = i / half, j = i - t * half;
        cs[t][j] = cos_sin(s_pos[t], p.rope.turn[j], p.rope.by);
    }
    __syncthreads();
    const int hq = p.q.p ? p.hq_s : 0, heads = hq + (p.k.p ? p.hkv_s : 0);
    const int per = p.d / 16, per_row = heads * per;
    for (int i = tid; i < n * per_row; i += kPgThreads) {
        const int t = i / per_row, in = i - t * per_row, h = in / per, u = in - h * per;
        const bool key = h >= hq;
        const TokenRows& x = key ? p.k : p.q;
        const int head = key ? h - hq : h, all = key ? p.hkv_s : p.hq_s;
        const T* src = static_cast<const T*>(x.p) + r * x.shard + (int64_t)(t0 + t) * x.token + head * p.d;
        T* dst = static_cast<T*>(key ? p.k_out : p.q_out) + (((int64_t)r * p.T + t0 + t) * all + head) * p.d;
        int at, bt;
        unit_at(p.rope, u, at, bt);
        float a[8], b[8];
        load8(src + at, a);
        load8(src + bt, b);
        turn_unit(p.rope, u, cs[t], a, b);
        store8(dst + at, a);
        store8(dst + bt, b);
    }
}

// ---------------------------------------------------------------------------

// Two float32 values as e4m3, to nearest even; what is not finite as NaN.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    uint32_t x = to_e4m3x2(lo, hi);
    if (!(fabsf(lo) < INFINITY)) x |= 0x7fu;
    if (!(fabsf(hi) < INFINITY)) x |= 0x7f00u;
    return x;
}
__device__ __forceinline__ uint2 e4m3x8(const float (&x)[8]) {
    return make_uint2(e4m3x2(x[0], x[1]) | e4m3x2(x[2], x[3]) << 16, e4m3x2(x[4], x[5]) | e4m3x2(x[6], x[7]) << 16);
}
__device__ __forceinline__ uint32_t requantise4(uint32_t x, float by) {
    uint32_t y = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float2 f = f16x2_to_float2(e4m3_to_f16x2((uint16_t)(x >> (16 * i))));
        y |= e4m3x2(f.x * by, f.y * by) << (16 * i);
    }
    return y;
}

// Largest magnitude of the finite bf16 of two words' halves.
__device__ __forceinline__ uint32_t max_finite(uint32_t m, uint32_t x) {
    x &= 0x7FFF7FFFu;
    return __vmaxu2(m, x & ~__vcmpgeu2(x, 0x7F807F80u));
}

// One CTA: the token rows of one window of a sequence, page-aligned positions
// of one page, for a shard: first the largest magnitude of every head's new
// keys and values, hence the scales; then what the page holds is brought to
// them where they grew; then the new rows, a few at a time with their sines.
//
// The windows are found without a pass over the batch: sequence b has those
// from cu[b] / page + 2 b on, of which it needs no more than there are before
// the next one's; where there are fewer rows than that, a row that begins a
// window has it.
__global__ void __launch_bounds__(kPgThreads) append_kernel(const __grid_constant__ AppendArgs p, int by_row) {
    __shared__ float2 cs[kPgRows][64];
    extern __shared__ uint32_t s_max[];                     // [2][hkv_s]: magnitudes of K and V, then 1 / scale
    const RopeArgs& a = p.r;
    const int tid = threadIdx.x, lane = tid & 31, hkv = a.hkv_s, d = a.d, page = p.c.page, per = d / 16;
    float* s_inv = reinterpret_cast<float*>(s_max);
    float* s_ratio = s_inv + 2 * hkv;                       // [2][hkv_s]: old scale over new one
    for (int i = tid; i < 2 * hkv; i += kPgThreads) s_max[i] = 0;
    if (cu_malformed(a.cu, a.B, a.T)) {
        if (tid == 0 && blockIdx.x == 0) set_status(a.status, TP_ERR_SHAPE);
        return;
    }
    const int r = blockIdx.x % a.N, slot = blockIdx.x / a.N, used = __ldg(a.cu + a.B), bits = 31 - __clz(page);
    int b, t0;
    int64_t w;                                              // the window: positions w page ..
    if (by_row) {
        if (slot >= used) return;
        b = sequence_of(a.cu, a.B, slot);
        t0 = slot;
        const int64_t pos = (int64_t)a.pos[b] + (t0 - a.cu[b]);
        w = pos >> bits;
        if (t0 != a.cu[b] && pos != w * page) return;
    } else {
        int lo = 0, hi = a.B;
        while (hi - lo > 1) {
            const int m = (lo + hi) >> 1;
            if ((__ldg(a.cu + m) >> bits) + 2 * m <= slot) lo = m;
            else hi = m;
        }
        b = lo;
        const int64_t k = slot - ((a.cu[b] >> bits) + 2 * b), pos = a.pos[b];
        w = (pos >> bits) + k;
        const int64_t row = a.cu[b] + (k ? w * page - pos : 0);
        if (row >= a.cu[b + 1]) return;
        t0 = (int)row;
    }
    const int64_t first = (int64_t)a.pos[b] + (t0 - a.cu[b]);          // position of row t0
    const int n = (int)min((int64_t)(a.cu[b + 1] - t0), (w + 1) * page - first), slot0 = (int)(first - w * page);
    int at = -1;                                                       // page of the pool
    if (w >= 0 && w < p.c.width) at = __ldg(p.c.pages + (int64_t)b * p.c.width + w);
    const bool there = at >= 0 && at < p.c.n_pages;
    if (!there && tid == 0) set_status(a.status, TP_ERR_CAPACITY);

    auto source = [&](const TokenRows& x, int t, int h) {
        return static_cast<const bf16*>(x.p) + r * x.shard + (int64_t)(t0 + t) * x.token + h * d;
    };
    auto stored = [&](int g) {                                         // head g's page, of K or (from hkv on) of V
        return (g < hkv ? p.c.k[r] : p.c.v[r]) + ((int64_t)at * hkv + (g < hkv ? g : g - hkv)) * page * d;
    };
    if (there) {
        const int vecs = d / 8, each = n * vecs, all = 2 * hkv * each; // 16-byte pieces, a head's together
        for (int i0 = 0; i0 < all; i0 += kPgThreads) {
            const int i = i0 + tid, g = min(i, all - 1) / each;
            uint32_t m = 0;
            if (i < all) {
                const int in = i - g * each, t = in / vecs, x = in - t * vecs;
                const uint4 v = *reinterpret_cast<const uint4*>(g < hkv ? source(a.k, t, g) + 8 * x : source(p.v, t, g - hkv) + 8 * x);
                m = max_finite(max_finite(max_finite(max_finite(0, v.x), v.y), v.z), v.w);
                m = max(m & 0xFFFFu, m >> 16);
            }
            const int g0 = __shfl_sync(0xffffffffu, g, 0);             // a warp's pieces are mostly one head's
            if (__all_sync(0xffffffffu, g == g0)) {
                m = __reduce_max_sync(0xffffffffu, m);
                if (lane == 0) atomicMax(&s_max[g], m);
            } else {
                atomicMax(&s_max[g], m);
            }
        }
        __syncthreads();
        for (int g = tid; g < 2 * hkv; g += kPgThreads) {
            float* scale = g < hkv ? p.c.ks[r] + (int64_t)at * hkv + g : p.c.vs[r] + (int64_t)at * hkv + g - hkv;
            const double x = (double)__uint_as_float(s_max[g] << 16) * (g < hkv ? p.k_growth : 1.0) / 448.0;
            // the least power of two not below x: x's exponent, and one more unless x is a power itself
            const long long word = __double_as_longlong(x);
            const int e = max(-60, (int)(word >> 52) - 1023 + ((word & 0xFFFFFFFFFFFFFll) != 0));
            float s = __uint_as_float((uint32_t)(127 + e) << 23), ratio = 1.f;
            if (slot0) {
                const float before = *scale;
                if (before > s) s = before;
                ratio = before / s;
            }
            *scale = s;
            s_inv[g] = 1.f / s;
            s_ratio[g] = ratio;
        }
        __syncthreads();
        const int old = slot0 * d / 16;                                // 16-byte pieces of what a head's page holds
        for (int g = 0; g < 2 * hkv; ++g) {
            const float ratio = s_ratio[g];
            if (!(ratio < 1.f)) continue;
            uint4* q = reinterpret_cast<uint4*>(stored(g));
            for (int i = tid; i < old; i += kPgThreads) {
                const uint4 v = q[i];
                q[i] = make_uint4(requantise4(v.x, ratio), requantise4(v.y, ratio), requantise4(v.z, ratio), requantise4(v.w, ratio));
            }
        }
    }

    const int half = a.rope.rot / 2, hq = a.q.p ? a.hq_s : 0, heads = hq + (there ? 2 * hkv : 0), per_row = heads * per;
    for (int r0 = 0; r0 < n; r0 += kPgRows) {
        const int rows = min(kPgRows, n - r0);
        if (half) {
            __syncthreads();
            for (int i = tid; i < rows * half; i += kPgThreads) {
                const int t = i / half, j = i - t * half;
                cs[t][j] = cos_sin(first + r0 + t, a.rope.turn[j], a.rope.by);
            }
            __syncthreads();
        }
        for (int i = tid; i < rows * per_row; i += kPgThreads) {
            const int t = i / per_row, in = i - t * per_row, h = in / per, u = in - h * per;
            const int g = h - hq;                                      // below 0: a query head
            const bool val = g >= hkv;
            const bf16* src = g < 0 ? source(a.q, r0 + t, h) : val ? source(p.v, r0 + t, g - hkv) : source(a.k, r0 + t, g);
            int x, y;
            if (val) x = 16 * u, y = x + 8;
            else unit_at(a.rope, u, x, y);
            float f[8], f2[8];
            load8(src + x, f);
            load8(src + y, f2);
            if (g >= 0) {                                              // by the scale first, so that no sum overflows
                const float inv = s_inv[g];
#pragma unroll
                for (int j = 0; j < 8; ++j) f[j] *= inv, f2[j] *= inv;
            }
            if (!val) turn_unit(a.rope, u, cs[t], f, f2);
            if (g < 0) {
                bf16* dst = static_cast<bf16*>(a.q_out) + (((int64_t)r * a.T + t0 + r0 + t) * a.hq_s + h) * d;
                store8(dst + x, f);
                store8(dst + y, f2);
            } else {
                uint8_t* dst = stored(g) + (slot0 + r0 + t) * d;
                const uint2 lo = e4m3x8(f), hi = e4m3x8(f2);
                if (y == x + 8) {
                    *reinterpret_cast<uint4*>(dst + x) = make_uint4(lo.x, lo.y, hi.x, hi.y);
                } else {
                    *reinterpret_cast<uint2*>(dst + x) = lo;
                    *reinterpret_cast<uint2*>(dst + y) = hi;
                }
            }
        }
    }
}

// ---------------------------------------------------------------------------

cudaError_t launch_rope(const RopeArgs& p, int dtype, cudaStream_t s) {
    RopeArgs a = p;
    // rows per CTA: as many as keep 8 CTAs per SM
    int rows = (int)((int64_t)a.T * a.N / (8 * kSMs));
    rows = rows < 1 ? 1 : rows > kPgRows ? kPgRows : rows;
    const int64_t ctas = (((int64_t)a.T + rows - 1) / rows) * a.N;
    if (ctas > INT32_MAX) return cudaErrorInvalidValue;
    if (dtype == TP_BF16) rope_kernel<bf16><<<(unsigned)ctas, kPgThreads, 0, s>>>(a, rows);
    else rope_kernel<float><<<(unsigned)ctas, kPgThreads, 0, s>>>(a, rows);
    return cudaGetLastError();
}

cudaError_t launch_append(const AppendArgs& p, cudaStream_t s) {
    AppendArgs a = p;
    const int64_t windows = a.r.T / a.c.page + 2 * (int64_t)a.r.B;
    const int by_row = a.r.T <= windows;
    const int64_t ctas = (by_row ? (int64_t)a.r.T : windows) * a.r.N;
    if (ctas > INT32_MAX) return cudaErrorInvalidValue;
    append_kernel<<<(unsigned)ctas, kPgThreads, 4 * a.r.hkv_s * sizeof(float), s>>>(a, by_row);
    return cudaGetLastError();
}

}  // namespace tpk
