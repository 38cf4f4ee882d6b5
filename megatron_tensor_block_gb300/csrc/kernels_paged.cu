// Rotary embedding of a packed batch, and appending its keys and values to
// 8-bit pages with that rotation on the way.
//
// A pair (a, b) of features turns by the angle p f: the host gives f as a
// 64-bit fraction of a turn per position, and p times it modulo 2^64 is the
// angle modulo a turn, exact for that f however far p is (a float32 product
// p f is off by whole degrees at p = 10^6). The nearest quarter turn is taken
// off as an integer; sine and cosine of the rest, at most an eighth of a turn,
// are their Taylor polynomials.
//
// A thread has sixteen features (eight pairs) of a token row and keeps their
// sines and cosines while it goes through heads. 16384 tokens of 32 query and 8
// KV heads of 128: 62 us on the device, 5.4 TB/s (with sines in shared memory
// for a shard's CTA, made again for every shard, 98; with frequencies from
// constant memory, which gives a warp's eight one after another, 63, and 49 for
// 36 in appending).
#include <climits>

#include "common.cuh"
#include "e4m3.cuh"
#include "paged.cuh"
#include "tp_internal.h"

namespace tpk {

constexpr int kPgThreads = 256, kPgAppend = 128;

// Whether cu is not 0 = cu[0] <= cu[1] <= ... <= T (the whole block asks).
__device__ __forceinline__ bool cu_malformed(const int* cu, int B, int T) {
    int bad = 0;
    for (int i = threadIdx.x; i < B; i += blockDim.x) bad |= cu_bad(cu, i, T);
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
    // the rest in 2^-62 quarters of a turn, within half of one: radians from its upper 32 bits (2^-32 of a quarter each)
    const float r = (float)(int)((int64_t)(x - (quarter << 62)) >> 30) * (1.5707963267948966f * 0x1p-32f), r2 = r * r;
    float s = fmaf(fmaf(fmaf(fmaf(2.7557319e-6f, r2, -1.9841270e-4f), r2, 8.3333333e-3f), r2, -1.6666667e-1f) * r2, r, r);
    float c = fmaf(fmaf(fmaf(fmaf(fmaf(-2.7557319e-7f, r2, 2.4801587e-5f), r2, -1.3888889e-3f), r2, 4.1666667e-2f), r2, -0.5f), r2, 1.f);
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
// The cosines and sines of unit u at position p. The frequencies are read from shared memory: a warp's lanes want different
// ones, which constant memory gives one after another.
__device__ __forceinline__ void unit_turns(const RopeTable& r, const uint64_t* turns, int u, int64_t p, float2 (&cs)[8]) {
    if (16 * u >= r.rot) return;
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        const ulonglong2 t = *reinterpret_cast<const ulonglong2*>(turns + 8 * u + i);
        cs[i] = cos_sin(p, t.x, r.by);
        cs[i + 1] = cos_sin(p, t.y, r.by);
    }
}
__device__ __forceinline__ void turn_unit(const RopeTable& r, int u, const float2 (&cs)[8], float (&a)[8], float (&b)[8]) {
    if (16 * u >= r.rot) return;
    if (r.layout == TP_ROPE_HALF) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float x = a[i], y = b[i];
            a[i] = x * cs[i].x - y * cs[i].y;
            b[i] = x * cs[i].y + y * cs[i].x;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
            const float2 t = cs[i / 2], v = cs[4 + i / 2];
            float x = a[i], y = a[i + 1];
            a[i] = x * t.x - y * t.y;
            a[i + 1] = x * t.y + y * t.x;
            x = b[i], y = b[i + 1];
            b[i] = x * v.x - y * v.y;
            b[i + 1] = x * v.y + y * v.x;
        }
    }
}

// Threads of a token row's units and of `split` groups of its heads of all shards, hq of q in each and then hk of k; a group's heads lie
// `split` apart, so that neighbouring threads have neighbouring memory. Bound by the bytes of the rows.
template <typename T>
__device__ __forceinline__ void rope_rows(const RopeArgs& p, const uint64_t* turns, int hq, int hk, int64_t thread, int split) {
    const int bits = p.d == 128 ? 3 : 2, u = (int)(thread & ((1 << bits) - 1));
    const int64_t rest = thread >> bits, row = rest <= INT_MAX ? (int)rest / split : rest / split;
    if (row >= __ldg(p.cu + p.B)) return;
    const int t = (int)row, b = sequence_of(p.cu, p.B, t);
    const int heads = p.N * (hq + hk);
    int x, y;
    unit_at(p.rope, u, x, y);
    float2 cs[8];
    unit_turns(p.rope, turns, u, (int64_t)__ldg(p.pos + b) + (t - __ldg(p.cu + b)), cs);
#pragma unroll 2
    for (int h = (int)(rest % split); h < heads; h += split) {
        const bool key = h >= p.N * hq;
        const int i = key ? h - p.N * hq : h, of = key ? hk : hq, r = i / of, head = i - r * of;
        const TokenRows& from = key ? p.k : p.q;
        const T* src = static_cast<const T*>(from.p) + r * from.shard + (int64_t)t * from.token + head * p.d;
        T* dst = static_cast<T*>(key ? p.k_out : p.q_out) + (((int64_t)r * p.T + t) * of + head) * p.d;
        float f[8], g[8];
        load8(src + x, f);
        load8(src + y, g);
        turn_unit(p.rope, u, cs, f, g);
        store8(dst + x, f);
        store8(dst + y, g);
    }
}

template <typename T>
__global__ void __launch_bounds__(kPgThreads) rope_kernel(const __grid_constant__ RopeArgs p, int split) {
    __shared__ __align__(16) uint64_t turns[64];
    if (threadIdx.x < 64) turns[threadIdx.x] = p.rope.turn[threadIdx.x];
    if (cu_malformed(p.cu, p.B, p.T)) {
        if (threadIdx.x == 0 && blockIdx.x == 0) set_status(p.status, TP_ERR_SHAPE);
        return;
    }
    rope_rows<T>(p, turns, p.q.p ? p.hq_s : 0, p.k.p ? p.hkv_s : 0, (int64_t)blockIdx.x * kPgThreads + threadIdx.x, split);
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
    float none = 0.f;                     // NaN where one of them is not finite, which is rare
#pragma unroll
    for (int i = 0; i < 8; ++i) none = fmaf(x[i], 0.f, none);
    if (none != none) return make_uint2(e4m3x2(x[0], x[1]) | e4m3x2(x[2], x[3]) << 16, e4m3x2(x[4], x[5]) | e4m3x2(x[6], x[7]) << 16);
    return make_uint2((uint32_t)to_e4m3x2(x[0], x[1]) | (uint32_t)to_e4m3x2(x[2], x[3]) << 16,
                      (uint32_t)to_e4m3x2(x[4], x[5]) | (uint32_t)to_e4m3x2(x[6], x[7]) << 16);
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
// them where they grew; then the new rows, which are in L1 by then. The
// queries' rows are CTAs of their own. Bound by the chain of a window's loads
// (offsets, rows and page, scale), some 6 us: 256 single tokens 9.4 us on the
// device, 24 prompts of 4695 tokens 32, of which their queries alone 14.8. With
// 256 threads to a window, of which fewer fit on an SM, 36.5.
//
// The windows are found without a pass over the batch: sequence b has those
// from cu[b] / page + 2 b on, of which it needs no more than there are before
// the next one's; where there are fewer rows than that, a row that begins a
// window has it.
__global__ void __launch_bounds__(kPgAppend, 6) append_kernel(const __grid_constant__ AppendArgs p, int by_row, int windows, int apart, int split) {
    __shared__ __align__(16) uint64_t turns[64];
    extern __shared__ uint32_t s_max[];                     // [2][hkv_s]: magnitudes of K and V, then 1 / scale
    const RopeArgs& a = p.r;
    const int tid = threadIdx.x, threads = blockDim.x, lane = tid & 31, hkv = a.hkv_s, d = a.d, page = p.c.page, per = d / 16;
    float* s_inv = reinterpret_cast<float*>(s_max);
    float* s_ratio = s_inv + 2 * hkv;                       // [2][hkv_s]: old scale over new one
    for (int i = tid; i < 2 * hkv; i += threads) s_max[i] = 0;
    if (tid < 64) turns[tid] = a.rope.turn[tid];
    if (cu_malformed(a.cu, a.B, a.T)) {
        if (tid == 0 && blockIdx.x == 0) set_status(a.status, TP_ERR_SHAPE);
        return;
    }
    // the CTAs of windows lie among those of queries, every `apart`-th: they wait for memory again and again, the others load it
    const int turn = blockIdx.x / apart, cta = min(turn, windows * a.N);
    if (turn * apart != (int)blockIdx.x || turn >= windows * a.N) {
        const int before = min(windows * a.N, turn + 1);
        rope_rows<bf16>(a, turns, a.hq_s, 0, (int64_t)((int)blockIdx.x - before) * threads + tid, split);
        return;
    }
    const int r = cta % a.N, slot = cta / a.N, used = __ldg(a.cu + a.B), bits = 31 - __clz(page);
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
    auto scale_of = [&](int g) { return g < hkv ? p.c.ks[r] + (int64_t)at * hkv + g : p.c.vs[r] + (int64_t)at * hkv + g - hkv; };
    auto source = [&](const TokenRows& x, int t, int h) {
        return static_cast<const bf16*>(x.p) + r * x.shard + (int64_t)(t0 + t) * x.token + h * d;
    };
    auto stored = [&](int g) {                                         // head g's page, of K or (from hkv on) of V
        return (g < hkv ? p.c.k[r] : p.c.v[r]) + ((int64_t)at * hkv + (g < hkv ? g : g - hkv)) * page * d;
    };
    // units of K and of V: the unit of a row fastest, then the row, then the head
    const int each = n * per, all = hkv * each, unit_bits = d == 128 ? 3 : 2;
    for (int i0 = 0; i0 < all; i0 += threads) {
        const int i = i0 + tid, h = min(i, all - 1) / each, in = min(i, all - 1) - h * each, t = in >> unit_bits, u = in & (per - 1);
        const uint4* k = reinterpret_cast<const uint4*>(source(a.k, t, h) + 16 * u);
        const uint4* v = reinterpret_cast<const uint4*>(source(p.v, t, h) + 16 * u);
        const uint4 x[4] = {k[0], k[1], v[0], v[1]};
        uint32_t m[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            uint32_t y = 0;
#pragma unroll
            for (int z = 2 * j; z < 2 * j + 2; ++z) y = max_finite(max_finite(max_finite(max_finite(y, x[z].x), x[z].y), x[z].z), x[z].w);
            m[j] = max(y & 0xFFFFu, y >> 16);
        }
        const int h0 = __shfl_sync(0xffffffffu, h, 0);                 // a warp's units are mostly one head's
        if (__all_sync(0xffffffffu, h == h0)) {
            m[0] = __reduce_max_sync(0xffffffffu, m[0]);
            m[1] = __reduce_max_sync(0xffffffffu, m[1]);
            if (lane < 2) atomicMax(&s_max[lane * hkv + h], lane ? m[1] : m[0]);
        } else {
            atomicMax(&s_max[h], m[0]);
            atomicMax(&s_max[hkv + h], m[1]);
        }
    }
    if (!there) {                                                      // (the rows' loads were on the way meanwhile)
        if (tid == 0) set_status(a.status, TP_ERR_CAPACITY);
        return;
    }
    float held = slot0 && tid < 2 * hkv ? *scale_of(tid) : 0.f;
    __syncthreads();
    bool grown = false;
    for (int g = tid; g < 2 * hkv; g += threads) {
        float* scale = scale_of(g);
        const double x = (double)__uint_as_float(s_max[g] << 16) * (g < hkv ? p.k_growth : 1.0) / 448.0;
        // the least power of two not below x: x's exponent, and one more unless x is a power itself
        const long long word = __double_as_longlong(x);
        // (127 at most, which is float32's end: only factors of the rotation above 158 ask for more)
        const int e = min(127, max(-60, (int)(word >> 52) - 1023 + ((word & 0xFFFFFFFFFFFFFll) != 0)));
        float s = __uint_as_float((uint32_t)(127 + e) << 23), ratio = 1.f;
        if (slot0) {
            const float before = g == tid ? held : *scale;
            if (before > s) s = before;
            ratio = before / s;
        }
        *scale = s;
        s_inv[g] = 1.f / s;
        s_ratio[g] = ratio;
        grown |= ratio < 1.f;
    }
    if (__syncthreads_or(grown)) {
        // 16-byte pieces of what a head's page holds before and behind the new rows
        const int row = d / 16, lo = slot0 * row, hi = (slot0 + n) * row, end = page * row;
        for (int g = 0; g < 2 * hkv; ++g) {
            const float ratio = s_ratio[g];
            if (!(ratio < 1.f)) continue;
            uint4* q = reinterpret_cast<uint4*>(stored(g));
            for (int i = tid; i < end; i += threads) {
                if (i >= lo && i < hi) continue;
                const uint4 v = q[i];
                q[i] = make_uint4(requantise4(v.x, ratio), requantise4(v.y, ratio), requantise4(v.z, ratio), requantise4(v.w, ratio));
            }
        }
    }
    for (int i = tid; i < all; i += threads) {
        const int h = i / each, in = i - h * each, t = in >> unit_bits, u = in & (per - 1);
        const float ki = s_inv[h], vi = s_inv[hkv + h];
        int x, y;
        unit_at(a.rope, u, x, y);
        const bf16* k = source(a.k, t, h);
        const bf16* v = source(p.v, t, h) + 16 * u;
        float f[8], g[8], f2[8], g2[8];
        load8(k + x, f);
        load8(k + y, g);
        load8(v, f2);
        load8(v + 8, g2);
        float2 cs[8];
        unit_turns(a.rope, turns, u, first + t, cs);
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] *= ki, g[j] *= ki, f2[j] *= vi, g2[j] *= vi;      // by the scale first, so that no sum overflows
        turn_unit(a.rope, u, cs, f, g);
        uint8_t* dst = stored(h) + (slot0 + t) * d;
        const uint2 lo = e4m3x8(f), hi = e4m3x8(g), lo2 = e4m3x8(f2), hi2 = e4m3x8(g2);
        if (y == x + 8) {
            *reinterpret_cast<uint4*>(dst + x) = make_uint4(lo.x, lo.y, hi.x, hi.y);
        } else {
            *reinterpret_cast<uint2*>(dst + x) = lo;
            *reinterpret_cast<uint2*>(dst + y) = hi;
        }
        *reinterpret_cast<uint4*>(stored(hkv + h) + (slot0 + t) * d + 16 * u) = make_uint4(lo2.x, lo2.y, hi2.x, hi2.y);
    }
}

// ---------------------------------------------------------------------------

// Groups of a row's heads: as many as give every SM 1024 threads, a head each at most.
static int rope_split(const RopeArgs& a, int64_t heads) {
    const int64_t rows = (int64_t)a.T * (a.d / 16), want = ((int64_t)kSMs * 1024 + rows - 1) / rows;
    return (int)(want < 1 ? 1 : want > heads ? heads : want);
}

cudaError_t launch_rope(const RopeArgs& p, int dtype, cudaStream_t s) {
    RopeArgs a = p;
    const int split = rope_split(a, (int64_t)a.N * ((a.q.p ? a.hq_s : 0) + (a.k.p ? a.hkv_s : 0)));
    const int64_t ctas = ((int64_t)a.T * (a.d / 16) * split + kPgThreads - 1) / kPgThreads;
    if (ctas > INT32_MAX) return cudaErrorInvalidValue;
    if (dtype == TP_BF16) rope_kernel<bf16><<<(unsigned)ctas, kPgThreads, 0, s>>>(a, split);
    else rope_kernel<float><<<(unsigned)ctas, kPgThreads, 0, s>>>(a, split);
    return cudaGetLastError();
}

cudaError_t launch_append(const AppendArgs& p, cudaStream_t s) {
    AppendArgs a = p;
    const int64_t most = a.r.T / a.c.page + 2 * (int64_t)a.r.B;
    const int by_row = a.r.T <= most;
    const int64_t windows = by_row ? (int64_t)a.r.T : most;
    const int threads = by_row ? 64 : kPgAppend, split = a.r.q.p ? rope_split(a.r, (int64_t)a.r.N * a.r.hq_s) : 0;
    const int64_t ctas = windows * a.r.N + ((int64_t)a.r.T * (a.r.d / 16) * split + threads - 1) / threads;
    if (ctas > INT32_MAX) return cudaErrorInvalidValue;
    append_kernel<<<(unsigned)ctas, threads, 4 * a.r.hkv_s * sizeof(float), s>>>(a, by_row, (int)windows, (int)(ctas / (windows * a.r.N)), split);
    return cudaGetLastError();
}

}  // namespace tpk
