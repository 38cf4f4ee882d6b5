// Attention of a packed batch over 8-bit pages.
//
//   o = sum_j w_j v_j / sum_j w_j,  w_j = 2^(s_j - m),  s_j = q . k_j log2(e) / sqrt(d)
//
// in one pass over the keys with a running m and sum.
#include <cfloat>
#include <cstring>
#include <mutex>

#include <cuda.h>
#include <cudaTypedefs.h>

#include "common.cuh"
#include "e4m3.cuh"
#include "paged.cuh"
#include "stream.cuh"
#include "tp_internal.h"

namespace tpk {

// ---------------------------------------------------------------------------
// Sequences of at most 32 query rows per KV head (rows: new tokens x heads of
// the group), in groups of 16: single tokens and a few drafted ones. Bound by the bytes of the
// pages, so the design keeps many of them on the way and gives every SM the
// same number.
//
// All the batch's chunks of 32 keys, sequence by sequence and head by head, are
// one list, cut into equal runs for the CTAs (one per SM) and each of those for
// its warps. Every CTA finds its place from the offsets and lengths by itself.
// A warp works alone: its own ring of stages in shared memory, no barrier with
// another warp but the one that copies until its run ends. What it has of a
// head that others have a part of is joined behind that, first in shared
// memory, then through the workspace by the CTA that comes last. One or two more
// warps copy, a lane for each of the others: page tables, scales, TMA boxes.
//
// Keys are the rows of the products, S^T = K Q^T and O^T = V^T P^T (16 x 8
// query rows), as fp16 x fp16: one conversion makes two fp16 of two e4m3,
// exactly; q is brought to fp16 by a power of two for each row, exactly but for
// elements below 2^-29 of the row's largest; the weights' rounding to fp16 is
// 2^-11. The scale of a page's keys goes into the scores, that of its values into
// the weights, relative to the row's largest weight times scale. (e4m3 x e4m3
// products of q in two terms, without conversions of K here: decode of 64 68 us
// where this took 63.)
//
// 128 single tokens over up to 16383 keys, 32 query and 8 KV heads of 128: 326 to
// 329 us on the device, 6.5 TB/s. 64 over 256 to 4095: 52 to 54, of which 1.7 pass
// until every warp has its place and 8 to 10 from the first CTA's last key to the
// last join. 32 of 1 to 8 tokens over 100 to 4000 keys in pages of 16: 71 (65 in
// larger ones).
// ---------------------------------------------------------------------------

constexpr float kPnRescale = 8.f;         // m and m + u follow their maxima where these have grown by more than this

struct PnPiece {                          // of a head of a sequence
    int64_t start;                        // the head's first chunk in the batch's list
    int h, x0, x1, nch;                   // chunks x0 .. x1 - 1 of nch; x1 = 0: none
    int c0, row0, rows, pos;              // the sequence's first token row, the rows of the head, its first position
};

// Fourteen warps and two that copy where no sequence has more than 8 rows, else eleven with more registers and one.
template <int D, int W>
struct PnShape {
    static constexpr int ROWS = W == 14 ? 8 : 16;
    static constexpr int TILE = kPnKeys * D;                        // bytes of a chunk's K or V
    static constexpr int STAGES = D == 128 ? 1 : 2;
    static constexpr int SLOT = ROWS * D * 4;                       // O of a piece of a head
    static constexpr int RING = STAGES * 2 * TILE;                  // of a warp
    static constexpr int COPIES = W == 14 ? 2 : 1;                  // warps that copy: for keys and for values, or half its lanes for either
    static constexpr int THREADS = 32 * (W + COPIES);
    struct Head {
        uint64_t kfull[W][STAGES], kempty[W][STAGES], vfull[W][STAGES], vempty[W][STAGES];
        float scales[W][STAGES][4];                                 // of K for both halves of the chunk, of V
        float4 mlu[2 * W][ROWS];                                    // (m, l, u) of the pieces
        int64_t sums[W + COPIES], firsts[W + COPIES];
        int64_t at[W];                                              // a warp's place in its first sequence
        PnPiece pieces[2 * W];                                      // of warp w: one that began before it, one that goes on behind it
        int valid[W][STAGES];                                       // halves whose page is there
        int seq[W], last[2], first_cta[2], many[W + COPIES], abort;
    };
    static constexpr int HEAD = ((int)sizeof(Head) + 1023) & ~1023;
    static constexpr int SMEM = HEAD + W * (RING + SLOT);
    static_assert(RING >= SLOT, "a warp's ring holds its last piece");
    static_assert(SMEM <= 227 * 1024, "shared memory");
};

struct PnArgs {
    CUtensorMap tk[TP_MAX_SHARDS], tv[TP_MAX_SHARDS];   // pools as [n_pages hkv_s][page][D] bytes, boxes of up to 32 keys
    const float* ks[TP_MAX_SHARDS];
    const float* vs[TP_MAX_SHARDS];
    const bf16* q;
    bf16* out;
    const int* cu;
    const int* pos;
    const int* pages;
    float* part_o;                        // [kSMs][2][rows][D], as the pieces in shared memory
    float4* part_mlu;                     // [kSMs][2][rows]
    unsigned* joined;                     // [kSMs] pieces of the head that begins in this CTA and ends in another
    int* status;
    int N, B, T, hq_s, hkv_s, G, bits, width, n_pages, max_new, cap, withheld;
    float scale_log2;
};

// Chunks of a sequence for each head: none where it is not this kernel's.
__device__ __forceinline__ int pn_chunks(const PnArgs& a, int b, int& c0, int& n, int& pos) {
    c0 = __ldg(a.cu + b);
    n = __ldg(a.cu + b + 1) - c0;
    pos = __ldg(a.pos + b);
    if (n <= 0 || n > a.max_new || (int64_t)n * a.G > kPnMost) return 0;
    return paged_chunks(n, pos, a.cap);
}

// A place in the batch's list of chunks: of a sequence, the chunks of every head's groups of rows.
struct PnCursor {
    int b, h, c, nch, c0, n, pos, groups; // h: head times groups, and the group
    __device__ __forceinline__ void begin(const PnArgs& a, int64_t in_sequence) {
        nch = pn_chunks(a, b, c0, n, pos);
        groups = paged_groups(n, a.G);
        h = (int)(in_sequence / nch);
        c = (int)(in_sequence - (int64_t)h * nch);
    }
    __device__ __forceinline__ void next(const PnArgs& a) {
        if (++c < nch) return;
        c = 0;
        if (++h < a.N * a.hkv_s * groups) return;
        h = 0;
        do {
            ++b;
            nch = b < a.B ? pn_chunks(a, b, c0, n, pos) : 1;
        } while (nch == 0);
        groups = paged_groups(n, a.G);
    }
    __device__ __forceinline__ int kend(const PnArgs& a) const {
        const int64_t end = (int64_t)pos + n;
        return (int)(end < 0 ? 0 : end > a.cap ? a.cap : end);
    }
};

__device__ __forceinline__ void mma_f16_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                              uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t at) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t at) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
}
__device__ __forceinline__ uint32_t movmatrix(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
// The power of two that brings a row's largest magnitude to 2^14 .. 2^15.
__device__ __forceinline__ float row_scale(float most) {
    const int e = (int)(__float_as_uint(most) >> 23);               // biased; 0: zero or subnormal, 255: infinite
    const int k = min(254, 127 + 14 + 127 - e);
    return most > 0.f ? __uint_as_float((uint32_t)k << 23) : 1.f;
}

// 16-byte unit u of row r of a tile, as the copies' swizzle puts it.
template <int D>
__device__ __forceinline__ uint32_t pn_unit(int r, int u) {
    if constexpr (D == 128) return r * 128 + ((u ^ (r & 7)) << 4);
    return r * 64 + ((u ^ ((r >> 1) & 3)) << 4);
}

// The copies of warp w's chunks, their keys and scales or (V) their values, by one lane, as its stages become free. Each copy is
// an instruction for each lane, one after another: a warp with the lanes of fifteen others' keys and values was the kernel's
// limit (128 long contexts 350 us, and 455 in pages of 16; 326 and 366 to 370 with a warp for either).
template <int D, int W>
__device__ __forceinline__ void pn_copies(const PnArgs& a, typename PnShape<D, W>::Head& hd, unsigned char* rings, int w, bool V, int64_t todo,
                                          int64_t in_sequence) {
    using Sh = PnShape<D, W>;
    constexpr int S = Sh::STAGES, TILE = Sh::TILE;
    const int page = 1 << a.bits;
    PnCursor at = {};
    if (todo > 0) {
        at.b = hd.seq[w];
        at.begin(a, in_sequence);
    }
    unsigned char* ring = rings + w * Sh::RING + (V ? TILE : 0);
    uint64_t* full = V ? &hd.vfull[w][0] : &hd.kfull[w][0];
    uint64_t* empty = V ? &hd.vempty[w][0] : &hd.kempty[w][0];
    uint32_t loads = 0;
    uint64_t since = global_ns();
    const uint64_t once = l2_evict_first_policy();
    while (__any_sync(0xffffffffu, todo > 0)) {
        const int s = loads % S;
        const bool go = todo > 0 && mbar_test(empty + s, ((loads / S) & 1) ^ 1);
        if (go) {
            const int key = kPnKeys * at.c, kend = at.kend(a), head = at.h / at.groups;
            const int shard = head / a.hkv_s, kv = head - shard * a.hkv_s;
            const int* row = a.pages + (int64_t)at.b * a.width;
            const bool in0 = key < kend, in1 = key + 16 < kend;
            const int id0 = in0 ? __ldg(row + (key >> a.bits)) : -1;
            const int id1 = in1 ? (a.bits == 4 ? __ldg(row + (key >> 4) + 1) : id0) : -1;
            const int mask = (id0 >= 0 && id0 < a.n_pages) | (id1 >= 0 && id1 < a.n_pages) << 1;
            const int tile0 = id0 * a.hkv_s + kv, tile1 = id1 * a.hkv_s + kv;
            if (!V) {
                if ((in0 && !(mask & 1)) || (in1 && !(mask & 2))) set_status(a.status, TP_ERR_CAPACITY);
                const uint32_t to = smem_u32(&hd.scales[w][s][0]);
                auto scale = [&](int i, const float* src) {
                    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(to + 4 * i), "l"(src) : "memory");
                };
                if (mask & 1) scale(0, a.ks[shard] + tile0), scale(2, a.vs[shard] + tile0);
                if (mask & 2) scale(1, a.ks[shard] + tile1), scale(3, a.vs[shard] + tile1);
                asm volatile("cp.async.mbarrier.arrive.noinc.shared.b64 [%0];" ::"r"(smem_u32(full + s)) : "memory");
                hd.valid[w][s] = mask;
            }
            const CUtensorMap* m = V ? &a.tv[shard] : &a.tk[shard];
            unsigned char* dst = ring + s * 2 * TILE;
            if (a.bits == 4) {                              // pages of 16: a box for each half
                mbar_arrive_expect_tx(full + s, __popc(mask) * (TILE / 2));
                if (mask & 1) tma_load_3d_hint(dst, m, 0, 0, tile0, full + s, once);
                if (mask & 2) tma_load_3d_hint(dst + TILE / 2, m, 0, 0, tile1, full + s, once);
            } else {
                mbar_arrive_expect_tx(full + s, (mask & 1) * TILE);
                if (mask & 1) tma_load_3d_hint(dst, m, 0, key & (page - 1), tile0, full + s, once);
            }
            ++loads;
            if (--todo > 0) at.next(a);
        }
        if (__any_sync(0xffffffffu, go)) {
            since = global_ns();
        } else {
            if (*(volatile int*)&hd.abort) break;
            if (global_ns() - since > 2 * kWaitLimitNs) {   // (the warps' own waits run out first)
                *(volatile int*)&hd.abort = 1;
                set_status(a.status, TP_ERR_TIMEOUT);
                break;
            }
            __nanosleep(32);
        }
    }
    // no copy may still be landing when the CTA exits, be it that another warp's wait runs out behind the last copy here
    volatile int no_abort = 0;
    for (uint32_t k = loads > S ? loads - S : 0; k < loads; ++k) mbar_wait(full + k % S, (k / S) & 1, &no_abort, nullptr);
}

template <int D, int W>
struct PnWarp {
    using Sh = PnShape<D, W>;
    const PnArgs& a;
    typename Sh::Head& hd;
    unsigned char* ring;                  // the warp's stages: K, then V
    int warp, lane;
    uint32_t done;                        // chunks worked on

    static constexpr int TILE = Sh::TILE, S = Sh::STAGES;

    __device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity) {
        return __all_sync(0xffffffffu, mbar_wait(bar, parity, &hd.abort, a.status));
    }
    __device__ __forceinline__ void release(uint64_t* bar) {
        __syncwarp();
        if (lane == 0) mbar_arrive(bar);
    }

    // The values of a chunk that some row does not see whole: what is not finite counts for the rows that see it (their sums
    // become NaN), and is taken out; so are the rows behind the last key. first: the chunk's first key.
    template <int NT>
    __device__ __forceinline__ void clean(unsigned char* v, int first, int kend, int there, const int (&lim)[NT][2], float (&o)[NT][D / 16][4]) {
        const bool gone = first + lane >= kend || !(there >> (lane >> 4) & 1);
        int found = 0;
        auto bad4 = [](uint32_t x) { return __vcmpeq4(x & 0x7F7F7F7Fu, 0x7F7F7F7Fu); };
#pragma unroll 1
        for (int u = 0; u < D / 16; ++u) {
            uint4* p = reinterpret_cast<uint4*>(v + pn_unit<D>(lane, u));
            if (gone) *p = make_uint4(0, 0, 0, 0);
            else {
                const uint4 x = *p;
                found |= (bad4(x.x) | bad4(x.y) | bad4(x.z) | bad4(x.w)) != 0;
            }
        }
        const unsigned rows = __ballot_sync(0xffffffffu, found);
        if (rows) {
            const int g = lane >> 2;
            for (int k = 0; k < kPnKeys; ++k) {
                if (!(rows >> k & 1)) continue;
#pragma unroll
                for (int mt = 0; mt < D / 16; ++mt) {
                    const unsigned char* p = v + pn_unit<D>(k, mt) + 2 * g;
                    const bool n0 = (p[0] & 0x7f) == 0x7f, n1 = (p[1] & 0x7f) == 0x7f;
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            if (n0 && first + k <= lim[nt][i]) o[nt][mt][i] = NAN;
                            if (n1 && first + k <= lim[nt][i]) o[nt][mt][2 + i] = NAN;
                        }
                }
            }
            __syncwarp();
            if (found)
#pragma unroll 1
                for (int u = 0; u < D / 16; ++u) {
                    uint4* p = reinterpret_cast<uint4*>(v + pn_unit<D>(lane, u));
                    const uint4 x = *p;
                    *p = make_uint4(x.x & ~bad4(x.x), x.y & ~bad4(x.y), x.z & ~bad4(x.z), x.w & ~bad4(x.w));
                }
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
    }

    // Whether there is a key up to lim in chunks w.x0 .. w.x1 - 1 (asked for rows without weights only).
    __device__ __forceinline__ bool sees(const PnCursor& cur, const PnPiece& w, int lim) const {
        const int end = (int)min((int64_t)lim + 1, (int64_t)kPnKeys * w.x1);
        for (int key = kPnKeys * w.x0; key < end; key += 16) {
            const int id = __ldg(a.pages + (int64_t)cur.b * a.width + (key >> a.bits));
            if (id >= 0 && id < a.n_pages) return true;
        }
        return false;
    }

    // Chunks w.x0 .. w.x1 - 1 of a head of the sequence at cur. Where that is all of them the result goes to out, else to
    // slot (O [rows][D] in units of 2^(m + u)) and (m, l, u) beside it.
    template <int NT>
    __device__ __forceinline__ bool head(const PnCursor& cur, const PnPiece& w, float* slot) {
        const int g = lane >> 2, t = lane & 3, kend = cur.kend(a);
        const int r = w.h / a.hkv_s, kvh = w.h - r * a.hkv_s;
        // the queries: rows 8 nt + g as columns of the products
        uint32_t qf[NT][D / 16][2];
        float factor[NT][2];
        int lim[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const bool is = 8 * nt + g < w.rows;
            const int row = w.row0 + 8 * nt + g, i = row / a.G;
            const bf16* src = a.q + (((int64_t)r * a.T + cur.c0 + i) * a.hq_s + kvh * a.G + (row - i * a.G)) * D + 4 * t;
            uint2 x[D / 16];
            float most = 0.f;
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks) {
                x[ks] = is ? *reinterpret_cast<const uint2*>(src + 16 * ks) : make_uint2(0, 0);
                const float2 f = unpack_bf16x2(x[ks].x), f2 = unpack_bf16x2(x[ks].y);
                most = fmaxf(fmaxf(most, fmaxf(fabsf(f.x), fabsf(f.y))), fmaxf(fabsf(f2.x), fabsf(f2.y)));
            }
            most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 1));
            most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 2));
            const float by = row_scale(most), back = a.scale_log2 / by;
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks) {
                const float2 f = unpack_bf16x2(x[ks].x), f2 = unpack_bf16x2(x[ks].y);
                qf[nt][ks][0] = pack_f16x2(f.x * by, f.y * by);
                qf[nt][ks][1] = pack_f16x2(f2.x * by, f2.y * by);
            }
#pragma unroll
            for (int i2 = 0; i2 < 2; ++i2) {
                const int mine = 8 * nt + 2 * t + i2, tok = (w.row0 + mine) / a.G;        // the lane's rows of S^T and O^T
                factor[nt][i2] = __shfl_sync(0xffffffffu, back, (2 * t + i2) * 4);
                const int64_t p = (int64_t)cur.pos + tok;
                lim[nt][i2] = mine < w.rows && p >= 0 && p < a.cap ? (int)p : -1;
            }
        }
        float o[NT][D / 16][4] = {}, m[NT][2], u[NT][2], l[NT][2];  // o holds O 2^-(m + u), l the sum of weights 2^(s - m)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 2; ++i) m[nt][i] = u[nt][i] = -INFINITY, l[nt][i] = 0.f;

        // the lane's row of a half's sixteen, and its first or second unit of two; units 2 i on: bits of the address exchanged
        const uint32_t unit = pn_unit<D>(lane & 15, lane >> 4);
        for (int c = w.x0; c < w.x1; ++c, ++done) {
            const int s = done % S;
            const uint32_t par = (done / S) & 1;
            unsigned char* kt = ring + s * 2 * TILE;
            const uint32_t at = smem_u32(kt) + unit;
            if (!wait(&hd.kfull[warp][s], par)) return false;
            float sc[NT][2][4], sl[1][2][4];                        // two sums for eight rows: shorter chains
#pragma unroll
            for (int kk = 0; kk < 2; ++kk) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int i = 0; i < 4; ++i) sc[nt][kk][i] = sl[0][kk][i] = 0.f;
#pragma unroll
                for (int ks = 0; ks < D / 16; ks += 2) {
                    uint32_t x[4];
                    // matrices: keys 0-7 and 8-15 of sixteen features, then of the next sixteen. A lane's four bytes are
                    // elements 2 t, 2 t + 1 and 2 t + 8, 2 t + 9 of the products' sum, as q is laid out too.
                    ldsm4(x, (at ^ (ks << 4)) + 16 * kk * D);
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const uint32_t a0 = e4m3_to_f16x2((uint16_t)x[2 * j]), a2 = e4m3_to_f16x2((uint16_t)(x[2 * j] >> 16));
                        const uint32_t a1 = e4m3_to_f16x2((uint16_t)x[2 * j + 1]), a3 = e4m3_to_f16x2((uint16_t)(x[2 * j + 1] >> 16));
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
                            mma_f16_16816(NT == 1 && j ? sl[0][kk] : sc[nt][kk], a0, a1, a2, a3, qf[nt][ks + j][0], qf[nt][ks + j][1]);
                    }
                }
            }
            const int there = *(volatile int*)&hd.valid[warp][s];
            const float4 pg = *reinterpret_cast<const float4*>(&hd.scales[warp][s][0]);
            const float pk[2] = {pg.x, pg.y};
            // of the values (a half that is not there: as the other, for its weights are 0)
            const float pv1 = there & 2 ? pg.w : there & 1 ? pg.z : 1.f, pv0 = there & 1 ? pg.z : pv1;
            const float lv[2] = {log2_of(pv0), log2_of(pv1)};
            release(&hd.kempty[warp][s]);

            const int first = kPnKeys * c;
            const bool whole = first + kPnKeys - 1 <= cur.pos && there == 3;   // every row sees every key
            float top[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float x[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int kk = j >> 1, e = i + 2 * (j & 1);
                        x[j] = (NT == 1 ? sc[nt][kk][e] + sl[0][kk][e] : sc[nt][kk][e]) * (factor[nt][i] * pk[kk]);
                        if (!whole) {
                            const int key = first + 16 * kk + 8 * (j & 1) + g;
                            if (key > lim[nt][i] || !(there >> kk & 1)) x[j] = -INFINITY;
                        }
                        sc[nt][kk][e] = x[j];
                    }
                    float y = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
                    y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 4));
                    y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 8));
                    top[nt][i] = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 16));
                }
            // A row's m follows the largest score, and m + u the largest of score and scale together, each where that has grown by
            // more than kPnRescale: only what the row sees counts, by its weight.
            bool moved = false;
            float m1[NT][2], u1[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const bool grow = top[nt][i] > m[nt][i] + kPnRescale;
                    m1[nt][i] = grow ? top[nt][i] : m[nt][i];
                    u1[nt][i] = grow ? u[nt][i] + (m[nt][i] - m1[nt][i]) : u[nt][i];
                    const float m0 = m1[nt][i] == -INFINITY ? 0.f : m1[nt][i];
                    float rise = (top[nt][i] - m0) + lv[0];
                    if (pv0 != pv1) {
                        rise = fmaxf((fmaxf(sc[nt][0][i], sc[nt][0][i + 2]) - m0) + lv[0], (fmaxf(sc[nt][1][i], sc[nt][1][i + 2]) - m0) + lv[1]);
                        rise = fmaxf(rise, __shfl_xor_sync(0xffffffffu, rise, 4));
                        rise = fmaxf(rise, __shfl_xor_sync(0xffffffffu, rise, 8));
                        rise = fmaxf(rise, __shfl_xor_sync(0xffffffffu, rise, 16));
                    }
                    const bool up = rise > u1[nt][i] + kPnRescale;
                    if (up) u1[nt][i] = rise;
                    moved |= grow || up;
                }
            if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const bool is = m1[nt][i] != m[nt][i] || u1[nt][i] != u[nt][i];
                        const float down = is ? m[nt][i] - m1[nt][i] : 0.f;                  // -inf at first
                        const float f = is ? ex2_approx(down + (u[nt][i] - u1[nt][i])) : 1.f;
                        if (is) l[nt][i] *= ex2_approx(down);
                        m[nt][i] = m1[nt][i];
                        u[nt][i] = u1[nt][i];
#pragma unroll
                        for (int mt = 0; mt < D / 16; ++mt) {
                            o[nt][mt][i] *= f;
                            o[nt][mt][2 + i] *= f;
                        }
                    }
            }
            uint32_t pb[NT][2][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const float b0 = m[nt][0] == -INFINITY ? 0.f : m[nt][0], b1 = m[nt][1] == -INFINITY ? 0.f : m[nt][1];
                const float u0 = u[nt][0] == -INFINITY ? 0.f : u[nt][0], u1 = u[nt][1] == -INFINITY ? 0.f : u[nt][1];
#pragma unroll
                for (int kk = 0; kk < 2; ++kk) {
                    // (an exponential for either: a weight can be below float32's smallest where its product with the scale counts)
                    float p[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float y = sc[nt][kk][e] - (e & 1 ? b1 : b0);
                        l[nt][e & 1] += ex2_approx(y);
                        p[e] = ex2_approx(y + (lv[kk] - (e & 1 ? u1 : u0)));
                    }
                    pb[nt][kk][0] = movmatrix(pack_f16x2(p[0], p[1]));
                    pb[nt][kk][1] = movmatrix(pack_f16x2(p[2], p[3]));
                }
            }
            if (!wait(&hd.vfull[warp][s], par)) return false;
            if (!whole) clean<NT>(kt + TILE, first, kend, there, lim, o);
#pragma unroll
            for (int kk = 0; kk < 2; ++kk)
#pragma unroll
                for (int mt = 0; mt < D / 16; mt += 2) {
                    uint32_t x[4];
                    // matrices: keys 0-7 and 8-15 of sixteen features, then of the next sixteen
                    ldsm4_t(x, (at ^ (mt << 4)) + TILE + 16 * kk * D);
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const uint32_t y0 = __byte_perm(x[2 * j], 0, 0x3120), y1 = __byte_perm(x[2 * j + 1], 0, 0x3120);
                        const uint32_t a0 = e4m3_to_f16x2((uint16_t)y0), a1 = e4m3_to_f16x2((uint16_t)(y0 >> 16));
                        const uint32_t a2 = e4m3_to_f16x2((uint16_t)y1), a3 = e4m3_to_f16x2((uint16_t)(y1 >> 16));
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) mma_f16_16816(o[nt][mt + j], a0, a1, a2, a3, pb[nt][kk][0], pb[nt][kk][1]);
                    }
                }
            release(&hd.vempty[warp][s]);
        }

        const bool all = w.x0 == 0 && w.x1 == w.nch;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float x = l[nt][i];
                x += __shfl_xor_sync(0xffffffffu, x, 4);
                x += __shfl_xor_sync(0xffffffffu, x, 8);
                x += __shfl_xor_sync(0xffffffffu, x, 16);
                const int row = 8 * nt + 2 * t + i;
                if (row >= w.rows) continue;
                const int of = w.row0 + row, tok = of / a.G;
                const int64_t p = (int64_t)cur.pos + tok;
                const bool none = p < 0 || p >= a.cap || (x == 0.f && !sees(cur, w, (int)p));      // no such place, no key seen: zeros
                if (all) {
                    const float half = ex2_approx(0.5f * u[nt][i]), f = half / x;           // (scores all -inf: 0 / 0)
                    bf16* dst = a.out + (((int64_t)r * a.T + cur.c0 + tok) * a.hq_s + kvh * a.G + (of - tok * a.G)) * D + 2 * g;
#pragma unroll
                    for (int mt = 0; mt < D / 16; ++mt)
                        *reinterpret_cast<uint32_t*>(dst + 16 * mt) =
                            none ? 0u : pack_bf16x2(o[nt][mt][i] * f * half, o[nt][mt][2 + i] * f * half);
                } else {
#pragma unroll
                    for (int mt = 0; mt < D / 16; ++mt)
                        *reinterpret_cast<float2*>(slot + row * D + 16 * mt + 2 * g) = make_float2(o[nt][mt][i], o[nt][mt][2 + i]);
                    // (a row that saw keys, whose scores were all -inf, has a finite m here: it is not one that saw none)
                    if (g == 0) hd.mlu[2 * warp + (w.x0 == 0)][row] = make_float4(none ? -INFINITY : fmaxf(m[nt][i], -FLT_MAX), x, u[nt][i], 0.f);
                }
            }
        return true;
    }
};

// One warp: a row's n pieces joined, l = sum_i 2^(m_i - m) l_i and, in units of
// 2^(m + u), o = sum_i 2^(m_i + u_i - m - u) o_i, always in the same order: no
// piece is as large as its values are, and none is lost whose weights are small
// but not its values. stat(i): (m, l, u) of piece i, read by lane i; get(i, x): the
// lane's D / 32 elements of its o. No piece is left out, so that a NaN of one
// stays. m is -inf where no piece has seen a key.
template <int D, typename Stat, typename Get>
__device__ __forceinline__ float4 pn_join(int n, int lane, Stat stat, Get get, float (&o)[D / 32]) {
    constexpr unsigned kAll = 0xffffffffu;
    constexpr int E = D / 32, AHEAD = 4;
    float m = -INFINITY, l = 0.f, u = -INFINITY;
#pragma unroll
    for (int k = 0; k < E; ++k) o[k] = 0.f;
    float x[AHEAD][E];
    auto load = [&](int i) {                                // on the way while the weights are found
#pragma unroll
        for (int j = 0; j < AHEAD; ++j)
            if (i + j < n) get(i + j, x[j]);
    };
    load(0);
#pragma unroll 1
    for (int i0 = 0; i0 < n; i0 += 32) {
        float4 s = make_float4(-INFINITY, 0.f, -INFINITY, 0.f);
        if (i0 + lane < n) s = stat(i0 + lane);
        const float top = fmaxf(m, warp_max(s.x)), m0 = top == -INFINITY ? 0.f : top;
        const float was = (m - m0) + u, its = (s.x - m0) + s.z;
        l = l * ex2_approx(m - m0) + warp_sum(s.y * ex2_approx(s.x - m0));
        m = top;
        u = fmaxf(was, warp_max(its));
        const float u0 = u == -INFINITY ? 0.f : u, down = ex2_approx(was - u0), w = ex2_approx(its - u0);
#pragma unroll
        for (int k = 0; k < E; ++k) o[k] *= down;
#pragma unroll 1
        for (int i = i0; i < min(i0 + 32, n); i += AHEAD) {
#pragma unroll
            for (int j = 0; j < AHEAD; ++j) {
                const float f = __shfl_sync(kAll, w, (i + j) & 31);
                if (i + j < n)
#pragma unroll
                    for (int k = 0; k < E; ++k) o[k] = fmaf(f, x[j][k], o[k]);
            }
            load(i + AHEAD);
        }
    }
    return make_float4(m, l, u, 0.f);
}

template <int D>
__device__ __forceinline__ void pn_store(const PnArgs& a, const PnPiece& p, int row, int lane, float4 mlu, const float (&o)[D / 32]) {
    const int r = p.h / a.hkv_s, kvh = p.h - r * a.hkv_s, of = p.row0 + row, tok = of / a.G;
    const int64_t at = (int64_t)p.pos + tok;
    const bool none = mlu.x == -INFINITY || at < 0 || at >= a.cap;
    bf16* dst = a.out + (((int64_t)r * a.T + p.c0 + tok) * a.hq_s + kvh * a.G + (of - tok * a.G)) * D + lane * (D / 32);
    const float half = ex2_approx(0.5f * mlu.z), f = half / mlu.y;          // (scores all -inf: 0 / 0)
    uint32_t y[D / 64];
#pragma unroll
    for (int k = 0; k < D / 64; ++k) y[k] = none ? 0u : pack_bf16x2(o[2 * k] * f * half, o[2 * k + 1] * f * half);
    if constexpr (D == 128) *reinterpret_cast<uint2*>(dst) = make_uint2(y[0], y[1]);
    else *reinterpret_cast<uint32_t*>(dst) = y[0];
}
template <int D>
__device__ __forceinline__ void pn_read(const float* src, int lane, float (&x)[D / 32], bool global) {
    if constexpr (D == 128) {
        const float4* p = reinterpret_cast<const float4*>(src) + lane;
        const float4 v = global ? __ldcg(p) : *p;
        x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
    } else {
        const float2* p = reinterpret_cast<const float2*>(src) + lane;
        const float2 v = global ? __ldcg(p) : *p;
        x[0] = v.x, x[1] = v.y;
    }
}

template <int D, int W>
__global__ void __launch_bounds__(PnShape<D, W>::THREADS, 1) paged_few_kernel(const __grid_constant__ PnArgs a) {
    using Sh = PnShape<D, W>;
    constexpr int S = Sh::STAGES, E = D / 32, THREADS = Sh::THREADS, WARPS = W + Sh::COPIES;
    extern __shared__ __align__(1024) unsigned char smem[];
    typename Sh::Head& hd = *reinterpret_cast<typename Sh::Head*>(smem);
    unsigned char* rings = smem + Sh::HEAD;
    unsigned char* slots = rings + W * Sh::RING;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        for (int i = 0; i < W * S; ++i) {
            mbar_init(&hd.kfull[0][0] + i, 2);               // the copies, and the scales
            mbar_init(&hd.kempty[0][0] + i, 1 + a.withheld);
            mbar_init(&hd.vfull[0][0] + i, 1);
            mbar_init(&hd.vempty[0][0] + i, 1);
        }
        hd.abort = (smem_u32(rings) & 1023u) ? 1 : 0;
        if (hd.abort) set_status(a.status, TP_ERR_ALIGN);
        fence_mbar_init();
    }
    if (tid < 2 * W) hd.pieces[tid].x1 = 0;
    if (tid < 2 * a.N) {
        const CUtensorMap* m = tid < a.N ? &a.tk[tid] : &a.tv[tid - a.N];
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(m)) : "memory");
    }
    pdl_trigger();
    pdl_wait();

    // ---- the CTA's and its warps' place in the list of chunks
    const int heads = a.N * a.hkv_s;
    int bad = 0, many = 0, off = 0;
    int64_t sum = 0, own = 0;                               // chunks of the thread's sequences, of the first of them
    for (int b = tid; b < a.B; b += THREADS) {
        int c0, n, pos;
        int64_t x = (int64_t)pn_chunks(a, b, c0, n, pos) * heads;
        if (x) x *= paged_groups(n, a.G);
        if (b == tid) own = x;
        sum += x;
        bad |= cu_bad(a.cu, b, a.T);
        many |= n > 0 && (int64_t)n * a.G > kPnMost && n <= a.max_new;
        if (n > a.max_new) off = TP_ERR_SHAPE;
        else if (n > 0 && !off && (pos < 0 || (int64_t)pos + n > a.cap)) off = TP_ERR_CAPACITY;
    }
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    int64_t upto_own = own;                                 // ... of those of the warp up to it
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xffffffffu, upto_own, o);
        if (lane >= o) upto_own += v;
    }
    many = __any_sync(0xffffffffu, many);
    if (lane == 0) hd.sums[warp] = sum, hd.many[warp] = many;
    if (lane == 31) hd.firsts[warp] = upto_own;
    if (__syncthreads_or(bad)) {
        if (tid == 0 && blockIdx.x == 0) set_status(a.status, TP_ERR_SHAPE);
        return;
    }
    if (blockIdx.x == 0 && off) set_status(a.status, off);
    int64_t total = 0, base = 0, before_own = upto_own - own;
    for (int i = 0; i < WARPS; ++i) {
        total += hd.sums[i];
        many |= hd.many[i];
        if (i < warp) before_own += hd.firsts[i];
        base += hd.firsts[i];
    }
    if (many && total <= kPagedFewBeside) return;        // left to the prompts' kernel
    // a chunk for each warp at least: fewer CTAs then have fewer pieces to join
    const int ctas = (int)min((int64_t)gridDim.x, (total + W - 1) / W);
    if ((int)blockIdx.x >= ctas) return;
    const int64_t from = total * blockIdx.x / ctas, upto = total * (blockIdx.x + 1) / ctas;
    // (a run for the first warps only where there are fewer chunks: the pieces of a head lie in warps next to one another)
    const int busy = (int)min((int64_t)W, upto - from);
    // lane w: the beginning of warp w's run
    const int64_t begin = from + (upto - from) * min(lane, busy) / busy;
    auto place = [&](int b, int64_t before, int64_t n) {     // whose run begins in one of the warp's sequences
        for (unsigned left = __ballot_sync(0xffffffffu, n && before < upto && before + n > from); left; left &= left - 1) {
            const int i = __ffs(left) - 1;
            const int64_t x = __shfl_sync(0xffffffffu, before, i), y = x + __shfl_sync(0xffffffffu, n, i);
            const int seq = __shfl_sync(0xffffffffu, b, i);
            if (lane < W && begin >= x && begin < y) {
                hd.seq[lane] = seq;
                hd.at[lane] = begin - x;
            }
        }
    };
    place(tid, before_own, own);
    for (int b0 = THREADS; b0 < a.B; b0 += THREADS) {
        const int b = b0 + tid;
        int c0, n, pos;
        int64_t x = b < a.B ? (int64_t)pn_chunks(a, b, c0, n, pos) * heads : 0;
        if (x) x *= paged_groups(n, a.G);
        int64_t y = x;
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t v = __shfl_up_sync(0xffffffffu, y, o);
            if (lane >= o) y += v;
        }
        __syncthreads();
        if (lane == 31) hd.firsts[warp] = y;
        __syncthreads();
        int64_t before = base + y - x;
        for (int i = 0; i < WARPS; ++i) {
            if (i < warp) before += hd.firsts[i];
            base += hd.firsts[i];
        }
        place(b, before, x);
    }
    __syncthreads();

    // ---- a warp's run
    constexpr unsigned kAll = 0xffffffffu;
    bool ok = !*(volatile int*)&hd.abort;
    if (warp >= W) {
        const int w = lane & 15;
        const int64_t first = __shfl_sync(kAll, begin, w), end = __shfl_sync(kAll, begin, w + 1);
        const bool v = Sh::COPIES == 2 ? warp > W : lane >= 16;
        const int64_t todo = w < W && ok && (Sh::COPIES == 1 || lane < 16) ? end - first : 0;
        pn_copies<D, W>(a, hd, rings, min(w, W - 1), v, todo, todo ? hd.at[w] : 0);
    } else {
        const int64_t w0 = __shfl_sync(kAll, begin, warp), w1 = __shfl_sync(kAll, begin, warp + 1);
        PnWarp<D, W> x{a, hd, rings + warp * Sh::RING, warp, lane, 0};
        PnCursor cur = {};
        if (w1 > w0) {
            cur.b = hd.seq[warp];
            cur.begin(a, hd.at[warp]);
        }
        int64_t at = w0;
        while (ok && at < w1) {
            PnPiece p;
            p.start = at - cur.c;
            p.h = cur.h / cur.groups;
            p.c0 = cur.c0;
            p.row0 = (cur.h - p.h * cur.groups) * kPnRows;
            p.rows = min(kPnRows, cur.n * a.G - p.row0);
            p.pos = cur.pos;
            p.x0 = cur.c;
            p.nch = cur.nch;
            p.x1 = (int)min((int64_t)cur.nch, cur.c + (w1 - at));
            const int second = p.x0 == 0;
            float* slot = reinterpret_cast<float*>(second ? rings + warp * Sh::RING : slots + warp * Sh::SLOT);
            if (Sh::ROWS == 8 || p.rows <= 8) ok = x.template head<1>(cur, p, slot);
            else ok = x.template head<Sh::ROWS / 8>(cur, p, slot);
            if (!ok) break;
            if (lane == 0 && !(p.x0 == 0 && p.x1 == p.nch)) hd.pieces[2 * warp + second] = p;
            at += p.x1 - p.x0;
            if (at < w1) {
                cur.c = cur.nch - 1;
                cur.next(a);
            }
        }
    }
    if (__syncthreads_or(!ok || *(volatile int*)&hd.abort)) return;

    // ---- pieces of a head, in this CTA: runs of pieces, which every warp finds by itself, their rows dealt out
    const PnPiece mine = hd.pieces[min(lane, 2 * W - 1)];
    const unsigned there = __ballot_sync(kAll, lane < 2 * W && mine.x1 > 0), below = there & ((1u << lane) - 1u);
    const int before = below ? 31 - __clz(below) : 0;
    const int64_t its = __shfl_sync(kAll, mine.start, before);
    const unsigned begins = __ballot_sync(kAll, (there >> lane & 1) && (!below || its != mine.start));
    auto slot_of = [&](int i) {
        return reinterpret_cast<const float*>(i & 1 ? rings + (i >> 1) * Sh::RING : slots + (i >> 1) * Sh::SLOT);
    };
    auto run_of = [&](int first, unsigned& pieces) {          // the run whose first piece it is
        const unsigned behind = begins & ~((2u << first) - 1u);
        pieces = there & ~((1u << first) - 1u) & (behind ? (1u << (__ffs(behind) - 1)) - 1u : kAll);
        PnPiece p = hd.pieces[first];
        p.x1 = hd.pieces[31 - __clz(pieces)].x1;
        return p;
    };
    const int stride = (int)min((int64_t)Sh::ROWS, (int64_t)a.max_new * a.G);
    for (int u = warp; u < __popc(begins) * stride; u += WARPS) {
        const int k = u / stride, row = u - k * stride;
        unsigned from_k = begins, pieces;
        for (int i = 0; i < k; ++i) from_k &= from_k - 1;
        // piece j of the run lies j places on: only a head's first piece is a warp's second one
        const int first = __ffs(from_k) - 1;
        const PnPiece p = run_of(first, pieces);
        if (row >= p.rows) continue;
        auto at = [&](int j) { return j ? ((first + 1) & ~1) + 2 * (j - (first & 1)) : first; };
        float o[E];
        const float4 r = pn_join<D>(
            __popc(pieces), lane, [&](int j) { return hd.mlu[at(j)][row]; },
            [&](int j, float (&x)[E]) { pn_read<D>(slot_of(at(j)) + row * D, lane, x, false); }, o);
        if (p.x0 == 0 && p.x1 == p.nch) {
            pn_store<D>(a, p, row, lane, r, o);
        } else {
            const int64_t dst = ((int64_t)blockIdx.x * 2 + (p.x0 == 0)) * Sh::ROWS + row;
            if (lane == 0) a.part_mlu[dst] = r;
            float* to = a.part_o + dst * D + lane * E;
            if constexpr (E == 4) *reinterpret_cast<float4*>(to) = make_float4(o[0], o[1], o[2], o[3]);
            else *reinterpret_cast<float2*>(to) = make_float2(o[0], o[1]);
        }
    }

    // ---- pieces of a head in several CTAs: the last of them joins. Only the CTA's first and last run can go on elsewhere.
    auto cta_of = [&](int64_t c) { return (int)(((c + 1) * ctas - 1) / total); };
    auto end_run = [&](int j, PnPiece& p) {
        if (begins == 0 || (j && !(begins & (begins - 1)))) return false;
        unsigned pieces;
        p = run_of(j ? 31 - __clz(begins) : __ffs(begins) - 1, pieces);
        return !(p.x0 == 0 && p.x1 == p.nch);
    };
    __threadfence();
    __syncthreads();
    if (tid < 2) {
        PnPiece p;
        int last = 0;
        if (end_run(tid, p)) {
            const int first = cta_of(p.start), n = cta_of(p.start + p.nch - 1) - first + 1;
            if (atomicAdd(a.joined + first, 1u) == (unsigned)n - 1) {
                a.joined[first] = 0;
                __threadfence();
                last = n;
                hd.first_cta[tid] = first;
            }
        }
        hd.last[tid] = last;
    }
    __syncthreads();
    for (int j = 0; j < 2; ++j) {
        const int n = hd.last[j], first = hd.first_cta[j];
        if (!n) continue;
        PnPiece p;
        end_run(j, p);
        auto src = [&](int i) { return ((int64_t)(first + i) * 2 + (i == 0)) * Sh::ROWS; };
        for (int row = warp; row < p.rows; row += WARPS) {
            float o[E];
            const float4 r = pn_join<D>(
                n, lane, [&](int i) { return __ldcg(a.part_mlu + src(i) + row); },
                [&](int i, float (&x)[E]) { pn_read<D>(a.part_o + (src(i) + row) * D, lane, x, true); }, o);
            pn_store<D>(a, p, row, lane, r, o);
        }
    }
}

// ---------------------------------------------------------------------------

cudaError_t byte_map(const void* base, int64_t d, int64_t d1, int64_t d2, int b1, int b2, CUtensorMap* out) {
    static std::mutex mu;
    static PFN_cuTensorMapEncodeTiled_v12000 encode = nullptr;
    {
        std::lock_guard<std::mutex> lock(mu);
        if (!encode) {
            cudaDriverEntryPointQueryResult q;
            cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", reinterpret_cast<void**>(&encode), 12000,
                                                             cudaEnableDefault, &q);
            if (e != cudaSuccess || !encode) return e != cudaSuccess ? e : cudaErrorNotSupported;
        }
    }
    cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)d1, (cuuint64_t)d2};
    cuuint64_t strides[2] = {(cuuint64_t)d, (cuuint64_t)(d1 * d)};
    cuuint32_t box[3] = {(cuuint32_t)d, (cuuint32_t)b1, (cuuint32_t)b2};
    cuuint32_t step[3] = {1u, 1u, 1u};
    const CUresult r = encode(out, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(base), dims, strides, box, step,
                              CU_TENSOR_MAP_INTERLEAVE_NONE, d == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

namespace {
constexpr size_t kPnMl = (size_t)kSMs * 2 * kPnRows * sizeof(float4);
size_t pn_part(int d) { return (size_t)kSMs * 2 * kPnRows * d * sizeof(float); }
}  // namespace

size_t paged_workspace(int64_t max_tokens, int heads, int group, int d) {
    return kPagedCtrl + kPnMl + pn_part(d) + (max_tokens * group <= kPnMost ? 0 : paged_wide_bytes(max_tokens, heads, d));
}

cudaError_t launch_attn_paged(const PagedAttnArgs& p, cudaStream_t s) {
    const int G = p.hq_s / p.hkv_s;
    const bool d128 = p.d == 128;
    {
        PnArgs a;
        memset(&a, 0, sizeof a);
        for (int r = 0; r < p.N; ++r) {
            const int64_t tiles = (int64_t)p.c.n_pages * p.hkv_s;
            const int rows = p.c.page < kPnKeys ? p.c.page : kPnKeys;
            cudaError_t e = byte_map(p.c.k[r], p.d, p.c.page, tiles, rows, 1, &a.tk[r]);
            if (e == cudaSuccess) e = byte_map(p.c.v[r], p.d, p.c.page, tiles, rows, 1, &a.tv[r]);
            if (e != cudaSuccess) return e;
            a.ks[r] = p.c.ks[r];
            a.vs[r] = p.c.vs[r];
        }
        a.q = static_cast<const bf16*>(p.q);
        a.out = static_cast<bf16*>(p.out);
        a.cu = p.cu;
        a.pos = p.pos;
        a.pages = p.c.pages;
        a.joined = reinterpret_cast<unsigned*>(p.ws + 256);
        a.part_mlu = reinterpret_cast<float4*>(p.ws + kPagedCtrl);
        a.part_o = reinterpret_cast<float*>(p.ws + kPagedCtrl + kPnMl);
        a.status = p.status;
        a.N = p.N;
        a.B = p.B;
        a.T = p.T;
        a.hq_s = p.hq_s;
        a.hkv_s = p.hkv_s;
        a.G = G;
        a.bits = 31 - __builtin_clz((unsigned)p.c.page);
        a.width = p.c.width;
        a.n_pages = p.c.n_pages;
        a.max_new = p.max_new;
        a.withheld = p.withheld;
        a.cap = p.c.width * p.c.page;
        a.scale_log2 = p.scale_log2;
        void* args[] = {&a};
        const bool eight = (int64_t)p.max_new * G <= 8;
        const void* fn = d128 ? (eight ? reinterpret_cast<const void*>(paged_few_kernel<128, 14>) : reinterpret_cast<const void*>(paged_few_kernel<128, 11>))
                              : (eight ? reinterpret_cast<const void*>(paged_few_kernel<64, 14>) : reinterpret_cast<const void*>(paged_few_kernel<64, 11>));
        const int smem = d128 ? (eight ? PnShape<128, 14>::SMEM : PnShape<128, 11>::SMEM) : (eight ? PnShape<64, 14>::SMEM : PnShape<64, 11>::SMEM);
        cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e == cudaSuccess) e = launch_pdl(fn, args, kSMs, smem, s, eight ? PnShape<64, 14>::THREADS : PnShape<64, 11>::THREADS);
        if (e != cudaSuccess) return e;
    }
    if ((int64_t)p.max_new * G <= kPnMost) return cudaSuccess;
    return launch_paged_wide(p, kPnMost, p.ws + kPagedCtrl + kPnMl + pn_part(p.d), s);
}

}  // namespace tpk
