// Attention over 8-bit pages of sequences that bring more than 32 query rows
// per KV head: prompts, and chunks of them; and the few of fewer rows beside
// them.
//
//   o = sum_j w_j v_j / sum_j w_j,  w_j = 2^(s_j - m),  s_j = q . k_j log2(e) / sqrt(d)
//
// in one pass over the keys with a running m and sum. An item is up to two
// tiles of 128 query rows (128 / G tokens of the G heads of a KV head) of a
// sequence; its keys come in blocks of 128. S = Q K^T and O += P V run on the
// tensor cores (tcgen05) with S, P and O in tensor memory:
//
// - S as e4m3 x e4m3: the keys' bytes go from their pages to the tensor cores as
//   they are (TMA, a box per page). Q, scaled by a power of two for each row, is
//   two e4m3 terms, which together have all of bf16's eight significant bits
//   (elements below 2^-10 of a row's largest are off by 2^-18 of it): twice the
//   products at twice the rate of 16-bit ones.
// - O += P V as fp16 x fp16: four warps widen a block's values to fp16, exactly,
//   and store them as the tensor cores read them; P is a weight times its page's
//   scale, relative to the row's largest such, and keeps 11 bits: the scale's
//   logarithm goes into the exponent. (P in two e4m3 terms would double what the
//   softmax warps do, which is most of what there is besides the products.)
//
// Bound by a tile's chain: its products, the softmax of 128 scores per thread,
// the hand-over, while the other tile's products take their turn. A block of
// 256 rows takes 3200 to 3300 cycles, 2048 of them products: a chunk of 512
// tokens behind 30001 keys, 32 query and 8 KV heads of 128, 187 to 195 us, 1.3 to
// 1.36 PFLOP/s. Short prompts pay 3 us for an item's beginning and end beside 1.7
// for a block (12 of up to 2048 tokens 65 to 68 us). Scales of values as factors of
// what is widened, over the item's largest so far, took 182 and 62 us, but lost
// bits of the values beside a page of a larger scale that a row does not see or
// that has no weight. Taken against: factors of a block read behind its scores without a
// group's lead (200 us), parts of four blocks at least (prompts 75 us where two
// took 72).
//
// The batch's blocks are one list, item by item, cut into equal runs for the
// CTAs, one per SM, each of which finds its place by itself. Parts of an item
// that two CTAs share are joined by a kernel behind this one.
//
// A kernel before this one writes q's terms (done here by the warps that widen
// values, an item's beginning waited 7 us for them). Warps: 0 copies, 1 and 2
// issue the products of a tile each, 3 walks the items and reads the page table
// and scales ahead, 4-11 softmax (four a tile), 12-15 widen values and write
// results.
#include <cfloat>
#include <cstring>

#include <cuda.h>

#include "attn.cuh"
#include "common.cuh"
#include "e4m3.cuh"
#include "paged.cuh"
#include "stream.cuh"
#include "tcgen05.cuh"
#include "tp_internal.h"

namespace tpk {

constexpr int kPwM = 128, kPwK = 128;     // query rows of a tile, keys of a block
constexpr int kPwThreads = 512;
constexpr int kPwQueue = 4;               // items read ahead
constexpr int kPwInfos = 12;              // blocks whose pages are read ahead, in fours
constexpr int kPwMinCut = 2;              // blocks of the shortest part of an item worth its join
constexpr int kPwCost = 3;                // what an item's beginning and end take, in blocks
constexpr float kPwRescale = 8.f;         // m and m + u follow their maxima where these have grown by more than this
constexpr float kPwFar = 40.f;            // binary orders between scales of values that one sum of weights is taken over
// Registers of the first four warps, the softmax's, and those that widen values: with 72, 168, 104 a chunk of 512 behind 30001 keys
// takes 192 us, with 64, 168, 112 189, with these 187; with 80, 168, 96 the last have most of theirs in memory.
constexpr int kPwRegsIo = 56, kPwRegsSoftmax = 168, kPwRegsOut = 120;
static_assert(kPwRegsIo + 2 * kPwRegsSoftmax + kPwRegsOut <= 4 * 128, "the launch's registers");

struct __align__(16) PwItem {
    int r, kvh, t0, ntok;                 // shard, KV head, first token row, tokens
    int b, qpos, kend, blk0;              // sequence, first token's position, end of its keys, first block
    int nb0, nb1, nb, nt;                 // blocks of the tiles and of both, tiles
    int part, end, poison, reserved;      // place of its partial results, or -1: final; 1: there are no more items; NaN among V
};
struct __align__(16) PwBlock {
    int tile[8];                          // per 16 keys: page and head, or -1: no key of it is seen
    float4 kl[4];                         // of two each: scale of the keys, times log2(e) / sqrt(d); log2 of the scale of the values
    float iv[8];                          // 2^(unit - that log2)
    float unit, lv_top;                   // that of the first page there of the item's part, a whole number; the block's largest lv
    int mask, far;                        // bit i: the 16 keys are there; their lv is more than kPwFar from unit (bit 8: of any so far)
};

template <int D>
struct PwShape {
    static constexpr int NKB = D / 64;
    static constexpr int QT = kPwM * D;                 // a term of a Q tile
    static constexpr int KB = kPwK * D;                 // a block of K or V in bytes
    static constexpr int VB = 2 * KB;                   // ... of V in fp16
    static constexpr int RK = D == 128 ? 3 : 6, RR = D == 128 ? 2 : 4, RV = D == 128 ? 2 : 3;
    struct Head {
        uint64_t q_full[2], q_empty[2], s_full[2], p_half[2], p_full[2], o_full[2], o_empty[2], st_full[2], st_empty[2], turn[2];
        uint64_t k_full[RK], k_empty[RK], r_full[RR], r_empty[RR], v_full[RV], v_empty[RV];
        uint64_t info_full[kPwInfos / 4], info_empty[kPwInfos / 4], item_full[kPwQueue], item_empty[kPwQueue], done;
        PwItem queue[kPwQueue];
        PwBlock info[kPwInfos];
        float2 stat[2][kPwM];                           // (m, l)
        float unit[2][kPwM];                            // u: O is in units of 2^(m + u)
        int64_t sums[3][kPwThreads / 32], start_at;
        int start_seq, abort;
        uint32_t tmem;
    };
    static constexpr int HEAD = ((int)sizeof(Head) + 1023) & ~1023;
    static constexpr int SMEM = HEAD + 4 * QT + RK * KB + RR * KB + RV * VB;
    static_assert(SMEM <= 227 * 1024, "shared memory");
};

struct PwArgs {
    CUtensorMap tq[2];                    // the terms of q as [N T][hq_s][D] bytes, boxes of a tile
    CUtensorMap tk[TP_MAX_SHARDS];        // pools as [n_pages hkv_s][page][D] bytes, boxes of a page
    const uint8_t* v[TP_MAX_SHARDS];
    const float* ks[TP_MAX_SHARDS];
    const float* vs[TP_MAX_SHARDS];
    const bf16* q;
    uint8_t* q_terms;                     // [2][N][T][hq_s][D]
    float* q_rows;                        // [N][T][hq_s] what a row's scores are multiplied by
    bf16* out;
    const int* cu;
    const int* pos;
    const int* pages;
    float* part_o;                        // [kSMs][2][256][D], in units of 2^(m + u)
    float4* part_mlu;                     // [kSMs][2][256]
    PagedCut* cuts;                       // [kSMs]
    int* status;
    int N, B, T, hq_s, hkv_s, G, tpt, bits, width, n_pages, max_new, cap, few, withheld;
    float scale_log2;
};

__device__ __forceinline__ int pw_blocks(const PwArgs& a, int pos, int tokens) {       // of keys before the end of the tokens
    const int64_t e = (int64_t)pos + tokens;
    return (int)(((e < 0 ? 0 : e > a.cap ? a.cap : e) + kPwK - 1) / kPwK);
}
// Units of a sequence for each head: its items' blocks, and what items take besides; 0 where it has `few` rows or fewer.
__device__ __forceinline__ int64_t pw_units(const PwArgs& a, int few, int b, int& c0, int& n, int& pos) {
    c0 = __ldg(a.cu + b);
    n = __ldg(a.cu + b + 1) - c0;
    pos = __ldg(a.pos + b);
    if (n <= 0 || n > a.max_new || (int64_t)n * a.G <= few) return 0;
    const int per = 2 * a.tpt;
    int64_t sum = 0;
    for (int i = 0; i < n; i += per) sum += pw_blocks(a, pos, min(n, i + per)) + kPwCost;
    return sum;
}

// D[tmem] (+)= A[smem] * B[smem]^T of bytes, 32 of the sum; every lane executes it, one issues.
__device__ __forceinline__ void mma_f8_w(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\tsetp.ne.b32 p, %4, 0;\n\telect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}
// e4m3 x e4m3 -> fp32, both K-major; fp16 x fp16 -> fp32, B MN-major.
__host__ __device__ constexpr uint32_t idesc_e4m3(int M, int N) {
    return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
__host__ __device__ constexpr uint32_t idesc_f16_bmn(int M, int N) { return idesc_e4m3(M, N) | (1u << 16); }

// A K-major tile of bytes with rows of D: swizzled over 128 bytes, or over 64.
template <int D>
__device__ __forceinline__ uint64_t byte_tile_desc(uint32_t saddr) {
    if constexpr (D == 128) return smem_desc_sw128(saddr);
    return (uint64_t)((saddr & 0x3FFFF) >> 4) | (uint64_t)1 << 16 | (uint64_t)(512 >> 4) << 32 | (uint64_t)1 << 46 | (uint64_t)4 << 61;
}
template <int D>
__device__ __forceinline__ uint32_t byte_tile_at(int r, int u) {           // 16-byte unit u of row r
    if constexpr (D == 128) return r * 128 + ((u ^ (r & 7)) << 4);
    return r * 64 + ((u ^ ((r >> 1) & 3)) << 4);
}

__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&v)[8]) {
    __syncwarp();
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(v[0]), "r"(v[1]), "r"(v[2]),
                 "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}
__device__ __forceinline__ uint32_t sub_f16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint16_t f16x2_to_e4m3x2(uint32_t x) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(x));
    return r;
}
__device__ __forceinline__ uint32_t e4m3_nan(uint32_t x) { return __vcmpeq4(x & 0x7F7F7F7Fu, 0x7F7F7F7Fu); }

__device__ __forceinline__ void bulk_copy(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(smem_u32(dst)), "l"(src),
                 "r"(bytes), "r"(smem_u32(bar))
                 : "memory");
}

template <int D>
__global__ void __launch_bounds__(kPwThreads, 1) paged_items_kernel(const __grid_constant__ PwArgs a) {
    using Sh = PwShape<D>;
    constexpr int RK = Sh::RK, RR = Sh::RR, RV = Sh::RV, WARPS = kPwThreads / 32;
    constexpr unsigned kAll = 0xffffffffu;
    extern __shared__ __align__(1024) unsigned char smem[];
    typename Sh::Head& hd = *reinterpret_cast<typename Sh::Head*>(smem);
    unsigned char* sq = smem + Sh::HEAD;                               // [2 tiles][2 terms]
    unsigned char* sk = sq + 4 * Sh::QT;
    unsigned char* sr = sk + RK * Sh::KB;                              // V as it comes
    unsigned char* sv = sr + RR * Sh::KB;                              // V in fp16
    volatile int* abort_flag = &hd.abort;
    const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;
    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&hd.q_full[i], 1);
            mbar_init(&hd.q_empty[i], 1);
            mbar_init(&hd.s_full[i], 1);
            mbar_init(&hd.p_half[i], 4);
            mbar_init(&hd.p_full[i], 4);
            mbar_init(&hd.o_full[i], 1);
            mbar_init(&hd.o_empty[i], 4);
            mbar_init(&hd.st_full[i], 4);
            mbar_init(&hd.st_empty[i], 4);
            mbar_init(&hd.turn[i], 1);
        }
        for (int i = 0; i < RK; ++i) mbar_init(&hd.k_full[i], 1), mbar_init(&hd.k_empty[i], 2 + a.withheld);
        for (int i = 0; i < RR; ++i) mbar_init(&hd.r_full[i], 1), mbar_init(&hd.r_empty[i], 4);
        for (int i = 0; i < RV; ++i) mbar_init(&hd.v_full[i], 4), mbar_init(&hd.v_empty[i], 2);
        for (int i = 0; i < kPwInfos / 4; ++i) mbar_init(&hd.info_full[i], 1), mbar_init(&hd.info_empty[i], 13);
        for (int i = 0; i < kPwQueue; ++i) mbar_init(&hd.item_full[i], 1), mbar_init(&hd.item_empty[i], 15);
        mbar_init(&hd.done, 2);
        hd.abort = (smem_u32(sq) & 1023u) ? 1 : 0;
        if (hd.abort) set_status(a.status, TP_ERR_ALIGN);
        fence_mbar_init();
    }
    if (warp == 1) tmem_alloc(smem_u32(&hd.tmem), 512);
    if (tid >= 64 && tid < 64 + a.N)
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&a.tk[tid - 64])) : "memory");
    pdl_trigger();
    pdl_wait();

    // ---- the CTA's place in the list of units
    const int heads = a.N * a.hkv_s;
    int bad = 0;
    int64_t sum[3] = {0, 0, 0}, own = 0, own_few = 0;       // units of the thread's sequences of many rows, and of few; the latter's chunks
    for (int b = tid; b < a.B; b += kPwThreads) {
        int c0, n, pos;
        const int64_t x = pw_units(a, 0, b, c0, n, pos) * heads;
        const bool few = (int64_t)n * a.G <= a.few;
        if (b == tid) own = few ? 0 : x, own_few = few ? x : 0;
        sum[0] += few ? 0 : x;
        sum[1] += few ? x : 0;
        if (few && x) sum[2] += paged_few_chunks(n, pos, a.G, a.cap) * heads;
        bad |= cu_bad(a.cu, b, a.T);
    }
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        for (int o = 16; o; o >>= 1) sum[i] += __shfl_xor_sync(kAll, sum[i], o);
        if (lane == 0) hd.sums[i][warp] = sum[i];
    }
    if (tid == 0) a.cuts[blockIdx.x].parts = 0;
    tc_fence_before();
    const bool malformed = __syncthreads_or(bad);
    tc_fence_after();
    const uint32_t tmem = uniform(hd.tmem);
    int64_t total = 0, total_few = 0, chunks = 0;
    if (!malformed)
        for (int i = 0; i < WARPS; ++i) total += hd.sums[0][i], total_few += hd.sums[1][i], chunks += hd.sums[2][i];
    // the sequences of few rows too, where the other kernel has left them
    const bool take = total > 0 && chunks <= kPagedFewBeside;
    const int few = take ? 0 : a.few;
    if (take) total += total_few, own += own_few;
    // parts of a few blocks at least: as few CTAs as that takes
    const int ctas = (int)min((int64_t)gridDim.x, (total + kPwMinCut + kPwCost - 1) / (kPwMinCut + kPwCost));
    const bool mine = (int)blockIdx.x < ctas;
    const int64_t from = mine ? total * blockIdx.x / ctas : 0, upto = mine ? total * (blockIdx.x + 1) / ctas : 0;
    if (mine) {
        int64_t base = 0;
        for (int b0 = 0; b0 < a.B; b0 += kPwThreads) {
            const int b = b0 + tid;
            int c0, n, pos;
            const int64_t x = b0 == 0 ? own : b < a.B ? pw_units(a, few, b, c0, n, pos) * heads : 0;
            int64_t y = x;
            for (int o = 1; o < 32; o <<= 1) {
                const int64_t v = __shfl_up_sync(kAll, y, o);
                if (lane >= o) y += v;
            }
            __syncthreads();
            if (lane == 31) hd.sums[0][warp] = y;
            __syncthreads();
            int64_t before = base + y - x;
            for (int i = 0; i < WARPS; ++i) {
                if (i < warp) before += hd.sums[0][i];
                base += hd.sums[0][i];
            }
            if (from >= before && from < before + x) {
                hd.start_seq = b;
                hd.start_at = before;
            }
        }
    }
    __syncthreads();

    auto item_done = [&](int k) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&hd.item_empty[k % kPwQueue]);
    };
    auto item_read = [&](int k, PwItem& w) {
        const int4* x = reinterpret_cast<const int4*>(&hd.queue[k % kPwQueue]);
        const int4 x0 = x[0], x1 = x[1], x2 = x[2];
        const int2 x3 = *reinterpret_cast<const int2*>(x + 3);
        w.r = x0.x, w.kvh = x0.y, w.t0 = x0.z, w.ntok = uniform(x0.w);
        w.b = x1.x, w.qpos = uniform(x1.y), w.kend = uniform(x1.z), w.blk0 = uniform(x1.w);
        w.nb0 = uniform(x2.x), w.nb1 = uniform(x2.y), w.nb = uniform(x2.z), w.nt = uniform(x2.w);
        w.part = x3.x, w.end = uniform(x3.y);
    };
    // the k-th item of the CTA; whether there is one. hold: the warp calls item_done itself
    auto item = [&](int k, PwItem& w, bool hold = false) {
        if (!__all_sync(kAll, mbar_wait(&hd.item_full[k % kPwQueue], (k / kPwQueue) & 1, abort_flag, a.status))) return false;
        item_read(k, w);
        if (!hold) item_done(k);
        return w.end == 0;
    };
    auto wait_all = [&](uint64_t* bar, uint32_t parity) {
        return (bool)__all_sync(kAll, at_wait(bar, parity, abort_flag, a.status));
    };
    // ... in the roles with other numbers of registers than the first: their waits have no call in them
    auto wait_in = [&](uint64_t* bar, uint32_t parity) {
        return (bool)__all_sync(kAll, mbar_wait(bar, parity, abort_flag, a.status));
    };
    // Entries of blocks are written and given back in fours; those of an item begin with a four.
    auto info_wait = [&](uint32_t n) { return wait_all(&hd.info_full[n / 4 % (kPwInfos / 4)], (n / kPwInfos) & 1); };
    auto info_wait_in = [&](uint32_t n) { return wait_in(&hd.info_full[n / 4 % (kPwInfos / 4)], (n / kPwInfos) & 1); };
    auto info_done = [&](uint32_t n) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&hd.info_empty[n / 4 % (kPwInfos / 4)]);
    };
    auto next_four = [](uint32_t n) { return (n + 3) & ~3u; };

    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kPwRegsIo));
        if (warp == 0) {
            // ---------------------------------------------------------------- loads
            uint32_t it = 0, iv = 0, n = 0, nq[2] = {0, 0}; // blocks of K and V, entries, Q tiles
            const int page = 1 << a.bits, step = page / 16, box = page * D;
            bool ok = !*abort_flag;
            PwItem w;
            for (int k = 0; ok && item(k, w); ++k, n = next_four(n)) {
                for (int j = 0; j < w.nb; ++j, ++n) {
                    if ((j & 3) == 0 && !(ok = info_wait(n))) break;
                    const int tile = hd.info[n % kPwInfos].tile[lane & 7];
                    const bool is = lane < 8 && lane % step == 0 && tile >= 0;
                    const uint32_t bytes = __popc(__ballot_sync(kAll, is)) * box;
                    const int s = it % RK, v = iv % RR;
                    if (!(ok = wait_all(&hd.k_empty[s], ((it / RK) & 1) ^ 1))) break;
                    if (lane == 0) mbar_arrive_expect_tx(&hd.k_full[s], bytes);
                    __syncwarp();
                    if (is) tma_load_3d_keep(sk + s * Sh::KB + lane * 16 * D, &a.tk[w.r], 0, 0, tile, &hd.k_full[s]);
                    ++it;
                    if (j == 0) {
#pragma unroll
                        for (int t = 0; t < 2; ++t) {
                            if (!ok || (t ? w.nb1 : w.nb0) == 0) continue;
                            if (!(ok = wait_all(&hd.q_empty[t], (nq[t] & 1) ^ 1))) continue;
                            ++nq[t];
                            if (lane == 0) {
                                mbar_arrive_expect_tx(&hd.q_full[t], 2 * a.tpt * a.G * D);
                                for (int x = 0; x < 2; ++x)
                                    tma_load_3d_keep(sq + (2 * t + x) * Sh::QT, &a.tq[x], 0, w.kvh * a.G, w.r * a.T + w.t0 + t * a.tpt,
                                                     &hd.q_full[t]);
                            }
                            __syncwarp();
                        }
                        if (!ok) break;
                    }
                    if (!(ok = wait_all(&hd.r_empty[v], ((iv / RR) & 1) ^ 1))) break;
                    if (lane == 0) mbar_arrive_expect_tx(&hd.r_full[v], bytes);
                    __syncwarp();
                    if (is) bulk_copy(sr + v * Sh::KB + lane * 16 * D, a.v[w.r] + (int64_t)tile * box, box, &hd.r_full[v]);
                    ++iv;
                    if ((j & 3) == 3 || j == w.nb - 1) info_done(n);
                }
            }
            volatile int no_abort = 0;                      // no copy may still be landing when the CTA exits
            if (lane == 0) {
                for (int t = 0; t < 2; ++t)
                    if (nq[t]) mbar_wait(&hd.q_full[t], (nq[t] - 1) & 1, &no_abort, nullptr);
                for (uint32_t i = it > RK ? it - RK : 0; i < it; ++i) mbar_wait(&hd.k_full[i % RK], (i / RK) & 1, &no_abort, nullptr);
                for (uint32_t i = iv > RR ? iv - RR : 0; i < iv; ++i) mbar_wait(&hd.r_full[i % RR], (i / RR) & 1, &no_abort, nullptr);
            }
        } else if (warp < 3) {
            // ---------------------------------------------------------------- products
            // A warp for each tile, which take turns, a block's products each. The whole warp runs the loop on warp-uniform
            // values and one elected lane issues.
            const int t = warp - 1;
            const uint32_t id_s = idesc_e4m3(kPwM, kPwK), id_o = idesc_f16_bmn(kPwM, D);
            const uint64_t dq = byte_tile_desc<D>(smem_u32(sq) + 2 * t * Sh::QT), dk0 = byte_tile_desc<D>(smem_u32(sk));
            const uint64_t dv0 = smem_desc_mn_sw128(smem_u32(sv), kPwK * 128, 1024);
            const uint32_t ts = tmem + kPwK * t, to = tmem + 2 * kPwK + D * t;
            uint32_t ik = 0, iv = 0, pp = 0, ip = 0, tp = 0;    // blocks of K and V, P, items of the tile, turns
            bool ok = !*abort_flag;
            auto take = [&]() { return wait_all(&hd.turn[t], (tp++ & 1) ^ (t == 0)); };
            auto pass = [&]() {
                if (lane == 0) mbar_arrive(&hd.turn[1 - t]);
                __syncwarp();
            };
            auto issue_s = [&](bool last) {                 // S = (Q1 + Q2) K^T
                const uint64_t dk = at_desc_add(dk0, ik % RK * Sh::KB);
#pragma unroll
                for (int x = 0; x < 2; ++x)
#pragma unroll
                    for (int i = 0; i < D / 32; ++i)
                        mma_f8_w(ts, at_desc_add(dq, x * Sh::QT + 32 * i), at_desc_add(dk, 32 * i), id_s, (x | i) != 0);
                tc_commit_w(smem_u32(&hd.s_full[t]));
                if (last) tc_commit_w(smem_u32(&hd.q_empty[t]));
            };
            auto issue_o = [&](bool first, int half) {      // O += P V, 64 of the 128 keys
                tc_mma4_ts_w(to, ts + 32 * half, at_desc_add(dv0, iv % RV * Sh::VB + 8192 * half), 8, 128, id_o, !first);
            };
            PwItem w;
            for (int k = 0; ok && item(k, w); ++k) {
                if (!w.nb) continue;
                const int n = t ? w.nb1 : w.nb0;
                if (!(ok = wait_all(&hd.k_full[ik % RK], (ik / RK) & 1))) break;
                if (n && !(ok = wait_all(&hd.q_full[t], ip & 1))) break;
                if (!(ok = take())) break;
                if (n) {
                    tc_fence_after();
                    issue_s(n == 1);
                }
                pass();
                tc_commit_w(smem_u32(&hd.k_empty[ik % RK]));
                ++ik;
                for (int j = 0; j < w.nb; ++j) {
                    const bool more = j + 1 < w.nb;
                    if (more && !(ok = wait_all(&hd.k_full[ik % RK], (ik / RK) & 1))) break;
                    if (!(ok = wait_all(&hd.v_full[iv % RV], (iv / RV) & 1))) break;
                    if (j < n) {
                        if (j == 0 && !(ok = wait_all(&hd.o_empty[t], (ip & 1) ^ 1))) break;
                        if (!(ok = wait_all(&hd.p_half[t], pp & 1))) break;
                    }
                    if (!(ok = take())) break;
                    if (j < n) {
                        tc_fence_after();
                        issue_o(j == 0, 0);
                        if (!(ok = wait_all(&hd.p_full[t], pp & 1))) break;
                        tc_fence_after();
                        issue_o(false, 1);
                        ++pp;
                        if (j + 1 == n) tc_commit_w(smem_u32(&hd.o_full[t]));
                    }
                    tc_commit_w(smem_u32(&hd.v_empty[iv % RV]));
                    ++iv;
                    if (j + 1 < n) issue_s(j + 2 == n);
                    pass();
                    if (more) {
                        tc_commit_w(smem_u32(&hd.k_empty[ik % RK]));
                        ++ik;
                    }
                }
                if (n) ++ip;
            }
            tc_commit_w(smem_u32(&hd.done));
        } else {
            // ---------------------------------------------------------------- items, and the pages of their blocks
            bool ok = !*abort_flag;
            int k = 0;
            uint32_t n = 0;
            auto publish = [&](const PwItem& w) {
                const int q = k % kPwQueue;
                if (!(ok = wait_all(&hd.item_empty[q], ((k / kPwQueue) & 1) ^ 1))) return;
                if (lane == 0) {
                    hd.queue[q] = w;
                    mbar_arrive(&hd.item_full[q]);
                }
                __syncwarp();
                ++k;
            };
            if (mine && ok) {
                int b = hd.start_seq, c0, len, pos;
                int64_t units = pw_units(a, few, b, c0, len, pos), at = hd.start_at;      // of the sequence for each head; the item's place
                int h = (int)((from - at) / units), i = 0;
                at += h * units;
                const int per = 2 * a.tpt;
                while (ok) {
                    const int ntok = min(per, len - i), nb = pw_blocks(a, pos, i + ntok);
                    const int64_t end = at + nb + kPwCost;
                    if (upto <= at) break;
                    // A cut inside an item: the block it falls before, none that leaves a part of fewer than kPwMinCut blocks;
                    // else the item is the next CTA's (0), or the last one's (-1).
                    auto block_at = [&](int64_t cut) {
                        const int64_t x = cut - at - kPwCost;
                        return nb < 2 * kPwMinCut || x < kPwMinCut ? 0 : nb - x < kPwMinCut ? -1 : (int)x;
                    };
                    const int lo = from <= at ? 0 : from >= end ? -1 : block_at(from);
                    const int cut = upto >= end ? -1 : block_at(upto);
                    if (lo >= 0) {
                        if (cut == 0) break;
                        const int hi = cut < 0 ? nb : cut;
                        PwItem w;
                        w.r = h / a.hkv_s;
                        w.kvh = h - w.r * a.hkv_s;
                        w.t0 = c0 + i;
                        w.ntok = ntok;
                        w.b = b;
                        w.qpos = (int)min((int64_t)pos + i, (int64_t)INT32_MAX);
                        const int64_t e = (int64_t)pos + i + ntok;
                        w.kend = (int)(e < 0 ? 0 : e > a.cap ? a.cap : e);
                        w.blk0 = lo;
                        w.nt = ntok > a.tpt ? 2 : 1;
                        w.nb0 = max(0, min(hi, pw_blocks(a, pos, i + min(ntok, a.tpt))) - lo);
                        w.nb1 = w.nt > 1 ? hi - lo : 0;
                        w.nb = max(w.nb0, w.nb1);
                        w.part = lo > 0 ? 0 : hi < nb ? 1 : -1;
                        w.end = w.poison = w.reserved = 0;
                        if (w.part == 1 && lane == 0) {
                            // CTAs with a cut inside the item: the next one on
                            const int64_t c = at + kPwCost;
                            const int last = (int)(((c + nb - kPwMinCut + 1) * ctas + total - 1) / total) - 1;
                            a.cuts[blockIdx.x] = PagedCut{last - (int)blockIdx.x + 1, w.t0, ntok, h, w.qpos};
                        }
                        publish(w);
                        if (!ok) break;
                        // pages of four blocks at a time: eight lanes for a block's sixteen keys each
                        float unit = 0.f;
                        bool any = false, wild = false;
                        for (int j = 0; j < w.nb; j += 4, n += 4) {
                            const int jj = j + (lane >> 3), g = lane & 7;
                            const int64_t key = (int64_t)(w.blk0 + jj) * kPwK + 16 * g;
                            int tile = -1;
                            float ks = 0.f, lv = 0.f;
                            if (jj < w.nb && key < w.kend) {
                                const int id = __ldg(a.pages + (int64_t)b * a.width + (int)(key >> a.bits));
                                if (id >= 0 && id < a.n_pages) {
                                    tile = id * a.hkv_s + w.kvh;
                                    ks = __ldg(a.ks[w.r] + tile);
                                    lv = log2_of(__ldg(a.vs[w.r] + tile));
                                } else {
                                    set_status(a.status, TP_ERR_CAPACITY);
                                }
                            }
                            __syncwarp();
                            const unsigned there = __ballot_sync(kAll, tile >= 0);
                            if (!any && there) {
                                unit = floorf(__shfl_sync(kAll, lv, __ffs(there) - 1));
                                any = true;
                            }
                            float lv_top = tile >= 0 ? lv : -INFINITY;
                            for (int o = 4; o; o >>= 1) lv_top = fmaxf(lv_top, __shfl_xor_sync(kAll, lv_top, o));
                            const unsigned far = __ballot_sync(kAll, tile >= 0 && fabsf(lv - unit) > kPwFar);
                            const unsigned upto_block = (2u << (lane | 7)) - 1u;     // (bit 31: all)
                            const int four = n / 4 % (kPwInfos / 4);
                            if (!(ok = wait_all(&hd.info_empty[four], ((n / kPwInfos) & 1) ^ 1))) break;
                            PwBlock& x = hd.info[(n + (lane >> 3)) % kPwInfos];
                            x.tile[g] = tile;
                            float* kl = reinterpret_cast<float*>(&x.kl[g >> 1]) + (g & 1);
                            kl[0] = ks * a.scale_log2;
                            kl[2] = lv;
                            x.iv[g] = tile >= 0 ? ex2_approx(fminf(unit - lv, 126.f)) : 1.f;
                            if (g == 0) {
                                x.unit = unit;
                                x.lv_top = lv_top;
                                x.mask = (int)(there >> (lane & 24) & 0xFFu);
                                x.far = (int)(far >> (lane & 24) & 0xFFu) | (wild || (far & upto_block) ? 0x100 : 0);
                            }
                            wild |= far != 0;
                            __syncwarp();
                            if (lane == 0) mbar_arrive(&hd.info_full[four]);
                        }
                        if (!ok || upto < end) break;
                    }
                    // the next item: of the sequence and head, of the next head, of the next sequence
                    at = end;
                    i += per;
                    if (i >= len) {
                        i = 0;
                        if (++h == heads) {
                            h = 0;
                            do {
                                units = ++b < a.B ? pw_units(a, few, b, c0, len, pos) : 1;
                            } while (units == 0);
                            if (b >= a.B) break;
                        }
                    }
                }
            }
            if (ok) {
                PwItem w = {};
                w.end = 1;
                publish(w);
            }
        }
    } else if (warp < 12) {
        // -------------------------------------------------------------------- softmax
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kPwRegsSoftmax));
        const int t = (warp - 4) >> 2;                      // tile
        const int qd = warp & 3;                            // tensor-memory lane quarter
        const int m = 32 * qd + lane;                       // row of the tile
        const int tok0 = m / a.G, tok = tok0 + t * a.tpt;   // the row's token in the item
        const uint32_t lane_off = (uint32_t)(32 * qd) << 16;
        const uint32_t s_col = tmem + lane_off + kPwK * t, o_col = tmem + lane_off + 2 * kPwK + D * t;
        uint32_t sp = 0, ip = 0, in = 0;                    // blocks, items of the tile, entries so far
        bool ok = !*abort_flag;
        PwItem w;
        for (int k = 0; ok && item(k, w); ++k) {
            const int n = t ? w.nb1 : w.nb0;
            const int rows = min(a.tpt, w.ntok - t * a.tpt) * a.G;
            const bool idle = 32 * qd >= rows;              // a warp without rows only keeps the barriers' pace
            const int own_max = (int)min((int64_t)w.kend - 1, (int64_t)w.qpos + tok);          // last key the row sees
            const int64_t warp_max = (int64_t)w.qpos + (32 * qd) / a.G + t * a.tpt;            // ... its warp's first row
            const int whole_to = (int)min(warp_max, (int64_t)w.kend - 1);
            // O is held in units of 2^(m + u), the sum of the weights 2^(s - m) in l. Both m and u are whole numbers.
            float m_use = -INFINITY, u_use = -INFINITY, l_run = 0.f;
            bool far = false, lost = false;                 // the row has seen a page far from the unit; keys, but no score above -inf
            const float factor = tok0 < a.tpt && tok < w.ntok ? __ldg(a.q_rows + ((int64_t)w.r * a.T + w.t0 + tok) * a.hq_s + w.kvh * a.G + m - tok0 * a.G) : 0.f;
            for (int j = 0; j < n; ++j, ++sp) {
                if ((j & 3) == 0 && !(ok = info_wait_in(in + j))) break;
                const PwBlock& x = hd.info[(in + j) % kPwInfos];
                // what the row's scores of sixteen keys each are multiplied by
                float kf[8];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 k = *reinterpret_cast<const float2*>(&x.kl[i]);
                    kf[2 * i] = k.x * factor;
                    kf[2 * i + 1] = k.y * factor;
                }
                const int key0 = (w.blk0 + j) * kPwK;
                // A block that every row of the warp sees whole needs no mask. (And below, s kf - m in one rounding is off by half
                // a step of m for the largest: scores so large that this counts are rounded before. S is below 2^24: the scores are
                // below 2^17 but for such factors.)
                const bool large = __any_sync(kAll, max3(max3(kf[0], kf[1], kf[2]), max3(kf[3], kf[4], kf[5]), fmaxf(kf[6], kf[7])) > 0x1p-7f);
                const bool whole = key0 + kPwK - 1 <= whole_to && x.mask == 0xFF && !large && !x.far;
                if (!(ok = wait_in(&hd.s_full[t], sp & 1))) break;
                if (!idle) {
                    tc_fence_after();
                    uint32_t v[4][32];
#pragma unroll
                    for (int c = 0; c < 4; ++c) tmem_ld32(s_col + 32 * c, v[c]);
                    float4 kl = x.kl[0];                    // of the first two sixteens
                    const float lv_top = x.lv_top;
                    tmem_wait_ld();
                    float* e = reinterpret_cast<float*>(&v[0][0]);
                    if (!whole) {
                        const int hi = own_max - key0, mask = x.mask;                // hi: last key of the block the row sees
#pragma unroll
                        for (int i = 0; i < 128; ++i) e[i] = i <= hi && (mask >> (i / 16) & 1) ? e[i] * kf[i / 16] : -INFINITY;
#pragma unroll
                        for (int i = 0; i < 8; ++i) kf[i] = 1.f;
                    }
                    auto top_of = [&](int c) {              // of sixteen keys
                        float y = fmaxf(e[16 * c], e[16 * c + 1]);
#pragma unroll
                        for (int i = 2; i < 16; i += 2) y = max3(y, e[16 * c + i], e[16 * c + i + 1]);
                        return y * kf[c];
                    };
                    float mq[4];                            // independent chains
#pragma unroll
                    for (int c = 0; c < 4; ++c) mq[c] = fmaxf(top_of(2 * c), top_of(2 * c + 1));
                    const float m_blk = fmaxf(fmaxf(mq[0], mq[1]), fmaxf(mq[2], mq[3]));
                    if (!whole) {
                        const int hi = own_max - key0, sees = hi < 0 ? 0 : x.mask & ((2 << (min(hi, kPwK - 1) >> 4)) - 1);
                        lost |= sees && m_blk == -INFINITY;
                        far |= (sees & x.far) != 0;
                    }
                    // m follows the largest score, m + u the largest of score and scale together that the row sees: what it does not
                    // see never reaches it. Mostly neither moves, which the largest scale of the block shows (seen or not).
                    float m_sub = m_use == -INFINITY ? 0.f : m_use;                  // nothing seen yet: every weight is 0
                    // (A row of NaN only is NaN as it is.)
                    if (__any_sync(kAll, m_blk > m_use + kPwRescale || (m_blk - m_sub) + lv_top > u_use + kPwRescale)) {
                        const bool grow = m_blk > m_use + kPwRescale;
                        const float m_new = grow ? floorf(m_blk) : m_use;
                        m_sub = m_new == -INFINITY ? 0.f : m_new;
                        float rise = -INFINITY, u_new = grow ? u_use + (m_use - m_new) : u_use;
#pragma unroll
                        for (int c = 0; c < 8; ++c) rise = fmaxf(rise, (top_of(c) - m_sub) + (c & 1 ? x.kl[c / 2].w : x.kl[c / 2].z));
                        if (rise > u_new + kPwRescale) u_new = floorf(rise);
                        const float by = m_new != m_use || u_new != u_use ? ex2_approx((m_use - m_new) + (u_use - u_new)) : 1.f;
                        if (grow) l_run *= ex2_approx(m_use - m_new);                // 0 when m_use is -inf
                        m_use = m_new;
                        u_use = u_new;
                        // O holds the blocks before this one (their products precede this S in the order of issue); rescale it
                        // where a row's unit moved
                        if (j > 0 && __any_sync(kAll, by != 1.f)) {
#pragma unroll 1
                            for (int c = 0; c < D / 8; ++c) {
                                uint32_t o[8];
                                tmem_ld8(o_col + 8 * c, o);
                                tmem_wait_ld();
#pragma unroll
                                for (int i = 0; i < 8; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * by);
                                tmem_st8(o_col + 8 * c, o);
                            }
                        }
                    }
                    const float u_sub = u_use == -INFINITY ? 0.f : u_use;
                    float base = -(m_sub + u_sub);
                    if (!whole) {                           // the scores themselves are there, in float32
                        base = -u_sub;
                        const uint64_t less = f2_pack(-m_sub, -m_sub);
#pragma unroll
                        for (int i = 0; i < 128; i += 2) f2_unpack(f2_add(f2_pack(e[i], e[i + 1]), less), e[i], e[i + 1]);
                        // The sum below is taken of weights times scales, each divided by its scale again: too far apart for float32
                        // where the scales are.
                        if (x.far) {
                            float sum = 0.f;
#pragma unroll
                            for (int i = 0; i < 128; ++i) sum += ex2_approx(e[i]);
                            if (far) l_run += sum;
                        }
                    }
                    uint64_t total = 0;
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        uint64_t scale2[2], add2[2], sum[2] = {0, 0};
#pragma unroll
                        for (int i = 0; i < 2; ++i) {       // (read again: registers)
                            const float k = whole ? (i ? kl.y : kl.x) * factor : 1.f, add = (i ? kl.w : kl.z) + base;
                            scale2[i] = f2_pack(k, k);
                            add2[i] = f2_pack(add, add);
                        }
                        const float2 back = *reinterpret_cast<const float2*>(&x.iv[2 * c]);
                        if (c < 3) kl = x.kl[c + 1];
                        uint32_t pk[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            float y, z;
                            f2_unpack(f2_fma(f2_pack(e[32 * c + 2 * i], e[32 * c + 2 * i + 1]), scale2[i / 8], add2[i / 8]), y, z);
                            y = ex2_approx(y);
                            z = ex2_approx(z);
                            sum[i / 8] = f2_add(sum[i / 8], f2_pack(y, z));
                            pk[i] = pack_f16x2(y, z);
                        }
#pragma unroll
                        for (int i = 0; i < 2; ++i) total = f2_fma(sum[i], i ? f2_pack(back.y, back.y) : f2_pack(back.x, back.x), total);
                        if (c == 2) {                       // the first 64 keys' products may begin
                            tmem_wait_st();
                            tc_fence_before();
                            __syncwarp();
                            if (lane == 0) mbar_arrive(&hd.p_half[t]);
                        }
                        tmem_st16(s_col + 16 * c, pk);
                    }
                    float sx, sy;
                    f2_unpack(total, sx, sy);
                    if (!far) l_run += (sx + sy) * ex2_approx((u_use == -INFINITY ? 0.f : u_use) - x.unit);
                    tmem_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&hd.p_full[t]);
                } else {
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(&hd.p_half[t]);
                        mbar_arrive(&hd.p_full[t]);
                    }
                }
                if ((j & 3) == 3 || j == w.nb - 1) info_done(in + j);
            }
            if (!ok) break;
            for (int j = n; j < w.nb; ++j)                  // blocks that only the other tile has
                if ((j & 3) == 3 || j == w.nb - 1) {
                    if (!(ok = info_wait_in(in + j))) break;
                    info_done(in + j);
                }
            if (!ok) break;
            in = next_four(in + w.nb);
            if (!n) continue;
            if (!(ok = wait_in(&hd.st_empty[t], (ip & 1) ^ 1))) break;
            // (a row that saw keys, whose scores were all -inf, has a finite m here: it is not one that saw none)
            hd.stat[t][m] = make_float2(l_run == 0.f && !lost ? -INFINITY : fmaxf(m_use, -FLT_MAX), l_run);
            hd.unit[t][m] = u_use;
            ++ip;
            __syncwarp();
            if (lane == 0) mbar_arrive(&hd.st_full[t]);
        }
    } else {
        // -------------------------------------------------------------------- values, results
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kPwRegsOut));
        const int qd = warp & 3, m = 32 * qd + lane;
        const int tok0 = m / a.G, g = m - tok0 * a.G;
        const uint32_t o_col = tmem + ((uint32_t)(32 * qd) << 16) + 2 * kPwK;
        uint32_t ip0 = 0, ip1 = 0, in = 0, ir = 0;
        bool ok = !*abort_flag;
        PwItem w;
        bool more = ok && item(0, w, true);
        for (int k = 0; ok && more; ++k) {
            // ---- values of the item's blocks, widened: a lane takes 16 bytes of a key, a warp 8 keys at a time. In a block that
            // some row does not see whole, NaN are taken out, to be put into the rows that see them at the end.
            int found = 0;
            for (int j = 0; j < w.nb; ++j, ++ir) {
                if ((j & 3) == 0 && !(ok = info_wait_in(in + j))) break;
                const int s = ir % RR, d = ir % RV;
                if (!(ok = wait_in(&hd.r_full[s], (ir / RR) & 1) && wait_in(&hd.v_empty[d], ((ir / RV) & 1) ^ 1))) break;
                const PwBlock& x = hd.info[(in + j) % kPwInfos];
                const int key0 = (w.blk0 + j) * kPwK, mask = x.mask;
                const bool ragged = (int64_t)key0 + kPwK > (int64_t)w.qpos + 1 || mask != 0xFF;
#pragma unroll 1
                for (int i = 0; i < 4; ++i) {
                    const int key = 32 * qd + 8 * i + (lane >> 2), u = lane & 3;
                    const bool gone = ragged && (key0 + key >= w.kend || !(mask >> (key >> 4) & 1));
#pragma unroll
                    for (int c0 = 0; c0 < Sh::NKB; ++c0) {
                        const int c = D == 128 ? c0 ^ (key & 1) : 0;                 // (halves of neighbours on other banks)
                        uint4 y = *reinterpret_cast<const uint4*>(sr + s * Sh::KB + key * D + 64 * c + 16 * u);
                        if (ragged) {
                            if (gone) y = make_uint4(0, 0, 0, 0);
                            const uint32_t n0 = e4m3_nan(y.x), n1 = e4m3_nan(y.y), n2 = e4m3_nan(y.z), n3 = e4m3_nan(y.w);
                            found |= (n0 | n1 | n2 | n3) != 0;
                            y = make_uint4(y.x & ~n0, y.y & ~n1, y.z & ~n2, y.w & ~n3);
                        }
                        const uint32_t in4[4] = {y.x, y.y, y.z, y.w};
                        uint32_t o[8];
#pragma unroll
                        for (int z = 0; z < 4; ++z) {
                            o[2 * z] = e4m3_to_f16x2((uint16_t)in4[z]);
                            o[2 * z + 1] = e4m3_to_f16x2((uint16_t)(in4[z] >> 16));
                        }
                        unsigned char* to = sv + d * Sh::VB + c * (kPwK * 128) + key * 128;
                        *reinterpret_cast<uint4*>(to + (((2 * u) ^ (key & 7)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
                        *reinterpret_cast<uint4*>(to + (((2 * u + 1) ^ (key & 7)) << 4)) = make_uint4(o[4], o[5], o[6], o[7]);
                    }
                }
                if (j == w.nb - 1 && __any_sync(kAll, found) && lane == 0) atomicOr(&hd.queue[k % kPwQueue].poison, 1);
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&hd.v_full[d]);
                    mbar_arrive(&hd.r_empty[s]);
                }
                if ((j & 3) == 3 || j == w.nb - 1) info_done(in + j);
            }
            if (!ok) break;
            in = next_four(in + w.nb);
            // ---- results
            const bool part = w.part >= 0;
            const int64_t prow = ((int64_t)blockIdx.x * 2 + (part ? w.part : 0)) * (2 * kPwM);
            char* base = part ? reinterpret_cast<char*>(a.part_o + prow * D)
                              : reinterpret_cast<char*>(a.out + (((int64_t)w.r * a.T + w.t0) * a.hq_s + w.kvh * a.G) * D);
            base += (lane & 3) * 16;
            int poison = 0;
#pragma unroll 1
            for (int t = 0; t < w.nt && ok; ++t) {
                const int n = t ? w.nb1 : w.nb0, tok = tok0 + t * a.tpt;
                const bool live = tok0 < a.tpt && tok < w.ntok;
                const int64_t pos = (int64_t)w.qpos + tok;
                float2 ml = make_float2(-INFINITY, 0.f);
                float u_row = -INFINITY;
                if (n) {
                    const uint32_t ph = (t ? ip1 : ip0) & 1;
                    if (!(ok = wait_in(&hd.st_full[t], ph) && wait_in(&hd.o_full[t], ph))) break;
                    if (t) ++ip1;
                    else ++ip0;
                    tc_fence_after();
                    ml = hd.stat[t][m];
                    u_row = hd.unit[t][m];
                }
                // (the item's last product, of the tile with most blocks, follows what all four warps have found)
                poison |= *reinterpret_cast<volatile int*>(&hd.queue[k % kPwQueue].poison);
                const bool zero = !n || (!part && (ml.x == -INFINITY || pos < 0 || pos >= a.cap));
                if (part && live) a.part_mlu[prow + t * kPwM + m] = make_float4(ml.x, ml.y, u_row, 0.f);
                const unsigned store = __ballot_sync(kAll, live) >> (lane & 28);
                const unsigned zeros = __ballot_sync(kAll, zero) >> (lane & 28);
                const int row = part ? (t * kPwM + m) * (D * 4) : (tok * a.hq_s + g) * (D * 2);
                int to[4];                                  // the four rows whose units the lane stores
#pragma unroll
                for (int i = 0; i < 4; ++i) to[i] = __shfl_sync(kAll, row, (lane & 28) | i);
                const uint32_t col = o_col + D * t;
                // 64 bytes of a row at a time, as four units; the next columns are read while these are written
                if (part) {
                    uint32_t o[16];
                    if (n) tmem_ld16(col, o);
#pragma unroll 1
                    for (int c = 0; c < D / 16; ++c) {
                        uint4 u[4] = {};
                        if (n) {
                            tmem_wait_ld();
#pragma unroll
                            for (int i = 0; i < 4; ++i) u[i] = make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
                            if (c + 1 < D / 16) tmem_ld16(col + 16 * c + 16, o);
                            transpose4(u, lane);
                        }
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (store >> i & 1) *reinterpret_cast<uint4*>(base + to[i] + 64 * c) = u[i];
                    }
                } else {
                    const float half = ex2_approx(0.5f * u_row), f = zero ? 0.f : half / ml.y;       // (scores all -inf: 0 / 0)
                    uint32_t o[32];
                    if (n) tmem_ld32(col, o);
#pragma unroll 1
                    for (int c = 0; c < D / 32; ++c) {
                        uint4 u[4] = {};
                        if (n) {
                            tmem_wait_ld();
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                u[i] = make_uint4(pack_bf16x2(__uint_as_float(o[8 * i]) * f * half, __uint_as_float(o[8 * i + 1]) * f * half),
                                                  pack_bf16x2(__uint_as_float(o[8 * i + 2]) * f * half, __uint_as_float(o[8 * i + 3]) * f * half),
                                                  pack_bf16x2(__uint_as_float(o[8 * i + 4]) * f * half, __uint_as_float(o[8 * i + 5]) * f * half),
                                                  pack_bf16x2(__uint_as_float(o[8 * i + 6]) * f * half, __uint_as_float(o[8 * i + 7]) * f * half));
                            if (c + 1 < D / 32) tmem_ld32(col + 32 * c + 32, o);
                            transpose4(u, lane);
                        }
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (store >> i & 1)
                                *reinterpret_cast<uint4*>(base + to[i] + 64 * c) = zeros >> i & 1 ? make_uint4(0, 0, 0, 0) : u[i];
                    }
                }
                if (n) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(&hd.o_empty[t]);
                        mbar_arrive(&hd.st_empty[t]);
                    }
                }
            }
            if (ok && __any_sync(kAll, poison)) {           // NaN among the values that a row sees
                __syncwarp();
                for (int t = 0; t < w.nt; ++t) {
                    const int tok = tok0 + t * a.tpt;
                    const int64_t pos = (int64_t)w.qpos + tok;
                    if (tok0 >= a.tpt || tok >= w.ntok || pos < 0 || pos >= a.cap) continue;
                    const int end = (int)min((int64_t)min(w.kend, (w.blk0 + w.nb) * kPwK) - 1, pos), page = 1 << a.bits;
                    const int* row = a.pages + (int64_t)w.b * a.width;
                    float* po = a.part_o + (prow + t * kPwM + m) * D;
                    bf16* out = a.out + (((int64_t)w.r * a.T + w.t0 + tok) * a.hq_s + w.kvh * a.G + g) * D;
                    // only blocks that NaN were taken out of, as above
#pragma unroll 1
                    for (int key0 = w.blk0 * kPwK; key0 <= end; key0 += kPwK) {
                        bool ragged = (int64_t)key0 + kPwK > (int64_t)w.qpos + 1;
                        for (int key = key0; !ragged && key < key0 + kPwK; key += page) {
                            const int id = __ldg(row + (key >> a.bits));
                            ragged = id < 0 || id >= a.n_pages;
                        }
                        if (!ragged) continue;
#pragma unroll 1
                        for (int key = key0; key < key0 + kPwK && key <= end; ++key) {
                            const int id = __ldg(row + (key >> a.bits));
                            if (id < 0 || id >= a.n_pages) continue;
                            const uint8_t* v = a.v[w.r] + (((int64_t)id * a.hkv_s + w.kvh) * page + (key & (page - 1))) * D;
#pragma unroll 1
                            for (int i = 0; i < D; i += 16) {
                                const uint4 x = *reinterpret_cast<const uint4*>(v + i);
                                if (!(e4m3_nan(x.x) | e4m3_nan(x.y) | e4m3_nan(x.z) | e4m3_nan(x.w))) continue;
                                for (int z = i; z < i + 16; ++z) {
                                    if ((v[z] & 0x7f) != 0x7f) continue;
                                    if (part) po[z] = NAN;
                                    else out[z] = __float2bfloat16_rn(NAN);
                                }
                            }
                        }
                    }
                }
            }
            if (!ok) break;
            item_done(k);
            more = item(k + 1, w, true);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        volatile int no_abort = 0;                   // every MMA has retired before the columns are freed
        mbar_wait(&hd.done, 0, &no_abort, nullptr);
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, 512);
        tmem_relinquish();
    }
}

// Rows of q in two e4m3 terms, scaled to 128 .. 256 by a power of two each: a lane takes sixteen features. Bound by its bytes.
template <int D>
__global__ void __launch_bounds__(256) paged_terms_kernel(const __grid_constant__ PwArgs a) {
    constexpr int LANES = D / 16;
    pdl_trigger();
    pdl_wait();
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, rows = (int64_t)a.N * a.T * a.hq_s;
    const bool is = i < rows * LANES;
    const uint4* src = reinterpret_cast<const uint4*>(a.q) + 2 * i;
    uint4 x[2];
#pragma unroll
    for (int z = 0; z < 2; ++z) x[z] = is ? __ldg(src + z) : make_uint4(0, 0, 0, 0);
    uint32_t most = 0;
#pragma unroll
    for (int z = 0; z < 2; ++z)
        most = __vmaxu2(__vmaxu2(__vmaxu2(most, x[z].x & 0x7FFF7FFFu), x[z].y & 0x7FFF7FFFu), __vmaxu2(x[z].z & 0x7FFF7FFFu, x[z].w & 0x7FFF7FFFu));
    most = max(most & 0xFFFFu, most >> 16);
#pragma unroll
    for (int o = 1; o < LANES; o <<= 1) most = max(most, __shfl_xor_sync(0xffffffffu, most, o));
    if (!is) return;
    const int e = (int)(most >> 7);                  // biased exponent of the row's largest magnitude
    // all of a row with infinities or NaN is NaN
    const float by = __uint_as_float((uint32_t)(e == 255 ? 255 : min(252, e ? 127 + 7 + 127 - e : 127)) << 23 | (e == 255));
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int v = 0; v < 4; ++v) {
        const uint4& y = x[v / 2];
        const float2 p = unpack_bf16x2(v & 1 ? y.z : y.x), q = unpack_bf16x2(v & 1 ? y.w : y.y);
        const uint32_t f[2] = {pack_f16x2(p.x * by, p.y * by), pack_f16x2(q.x * by, q.y * by)};
        uint32_t h[2], l[2];
#pragma unroll
        for (int z = 0; z < 2; ++z) {
            h[z] = f16x2_to_e4m3x2(f[z]);
            l[z] = f16x2_to_e4m3x2(sub_f16x2(f[z], e4m3_to_f16x2((uint16_t)h[z])));
        }
        hi[v] = h[0] | h[1] << 16;
        lo[v] = l[0] | l[1] << 16;
    }
    uint4* dst = reinterpret_cast<uint4*>(a.q_terms);
    dst[i] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    dst[rows * LANES + i] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    if (i % LANES == 0) a.q_rows[i / LANES] = e == 255 ? 1.f : 1.f / by;
}

// Rows of the items that were cut, a warp each, over the parts in their order: l = sum_i 2^(m_i - m) l_i and, in units of
// 2^(m + u), o = sum_i 2^(m_i + u_i - m - u) O_i: no part is as large as its values are, and none is lost whose weights are
// small but not its values. No part is left out, so that a NaN of one stays. m is -inf where no part has seen a key.
template <int D>
__global__ void __launch_bounds__(128) paged_join_kernel(const __grid_constant__ PwArgs a, int slices) {
    constexpr int E = D / 32, AHEAD = 4;             // elements per lane, parts loaded together
    pdl_trigger();
    pdl_wait();
    const int cta = blockIdx.x / slices, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const PagedCut c = a.cuts[cta];
    for (int row = (blockIdx.x - cta * slices) * 4 + warp; c.parts && row < 2 * kPwM; row += 4 * slices) {
        const int t = row / kPwM, m = row - t * kPwM, tok0 = m / a.G, tok = tok0 + t * a.tpt;
        if (tok0 >= a.tpt || tok >= c.ntok) continue;
        const int r = c.h / a.hkv_s, kvh = c.h - r * a.hkv_s;
        // the first part is the second place of the CTA that begins the item, the others the first places of those behind it
        auto place = [&](int i) { return ((int64_t)(cta + i) * 2 + (i == 0)) * (2 * kPwM) + row; };
        float top = -INFINITY, l = 0.f, u = -INFINITY, o[E] = {};
        for (int i0 = 0; i0 < c.parts; i0 += AHEAD) {
            float4 s[AHEAD];
            float x[AHEAD][E];
#pragma unroll
            for (int i = 0; i < AHEAD; ++i) {
                if (i0 + i >= c.parts) break;
                s[i] = __ldcg(a.part_mlu + place(i0 + i));
                const float* src = a.part_o + place(i0 + i) * D + lane * E;
                if constexpr (E == 4) {
                    const float4 y = __ldcg(reinterpret_cast<const float4*>(src));
                    x[i][0] = y.x, x[i][1] = y.y, x[i][2] = y.z, x[i][3] = y.w;
                } else {
                    const float2 y = __ldcg(reinterpret_cast<const float2*>(src));
                    x[i][0] = y.x, x[i][1] = y.y;
                }
            }
#pragma unroll
            for (int i = 0; i < AHEAD; ++i) {
                if (i0 + i >= c.parts) break;
                const float m2 = fmaxf(top, s[i].x), m0 = m2 == -INFINITY ? 0.f : m2;
                const float was = (top - m0) + u, its = (s[i].x - m0) + s[i].z;
                l = l * ex2_approx(top - m0) + s[i].y * ex2_approx(s[i].x - m0);
                top = m2;
                u = fmaxf(was, its);
                const float u0 = u == -INFINITY ? 0.f : u, f = ex2_approx(was - u0), w = ex2_approx(its - u0);
#pragma unroll
                for (int e = 0; e < E; ++e) o[e] = o[e] * f + x[i][e] * w;
            }
        }
        const int64_t pos = (int64_t)c.qpos + tok;
        const bool none = top == -INFINITY || pos < 0 || pos >= a.cap;
        const float half = ex2_approx(0.5f * u), f = half / l;             // (scores all -inf: 0 / 0)
        uint32_t y[E / 2];
#pragma unroll
        for (int e = 0; e < E / 2; ++e) y[e] = none ? 0u : pack_bf16x2(o[2 * e] * f * half, o[2 * e + 1] * f * half);
        bf16* dst = a.out + (((int64_t)r * a.T + c.t0 + tok) * a.hq_s + kvh * a.G + (m - tok0 * a.G)) * D + lane * E;
        if constexpr (E == 4) *reinterpret_cast<uint2*>(dst) = make_uint2(y[0], y[1]);
        else *reinterpret_cast<uint32_t*>(dst) = y[0];
    }
}

// Cuts, partial (m, l, u), partial O, q's terms and rows.
static size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }
static const size_t kPwCuts = up256(kSMs * sizeof(PagedCut)), kPwMl = (size_t)kSMs * 2 * 2 * kPwM * sizeof(float4);
static size_t pw_o(int d) { return (size_t)kSMs * 2 * 2 * kPwM * d * sizeof(float); }
size_t paged_wide_bytes(int64_t tokens, int heads, int d) {
    return kPwCuts + kPwMl + pw_o(d) + up256((size_t)tokens * heads * d * 2) + up256((size_t)tokens * heads * sizeof(float));
}

cudaError_t launch_paged_wide(const PagedAttnArgs& p, int few, char* ws, cudaStream_t s) {
    PwArgs a;
    memset(&a, 0, sizeof a);
    a.cuts = reinterpret_cast<PagedCut*>(ws);
    a.part_mlu = reinterpret_cast<float4*>(ws + kPwCuts);
    a.part_o = reinterpret_cast<float*>(ws + kPwCuts + kPwMl);
    a.q_terms = reinterpret_cast<uint8_t*>(ws + kPwCuts + kPwMl + pw_o(p.d));
    const int64_t rows = (int64_t)p.N * p.T * p.hq_s;
    a.q_rows = reinterpret_cast<float*>(a.q_terms + up256((size_t)rows * p.d * 2));
    const int G = p.hq_s / p.hkv_s;
    for (int x = 0; x < 2; ++x) {
        const cudaError_t e = byte_map(a.q_terms + x * rows * p.d, p.d, p.hq_s, (int64_t)p.N * p.T, G, kPwM / G, &a.tq[x]);
        if (e != cudaSuccess) return e;
    }
    for (int r = 0; r < p.N; ++r) {
        const cudaError_t e = byte_map(p.c.k[r], p.d, p.c.page, (int64_t)p.c.n_pages * p.hkv_s, p.c.page, 1, &a.tk[r]);
        if (e != cudaSuccess) return e;
        a.v[r] = p.c.v[r];
        a.ks[r] = p.c.ks[r];
        a.vs[r] = p.c.vs[r];
    }
    a.q = static_cast<const bf16*>(p.q);
    a.out = static_cast<bf16*>(p.out);
    a.cu = p.cu;
    a.pos = p.pos;
    a.pages = p.c.pages;
    a.status = p.status;
    a.N = p.N;
    a.B = p.B;
    a.T = p.T;
    a.hq_s = p.hq_s;
    a.hkv_s = p.hkv_s;
    a.G = G;
    a.tpt = kPwM / a.G;
    a.bits = 31 - __builtin_clz((unsigned)p.c.page);
    a.width = p.c.width;
    a.n_pages = p.c.n_pages;
    a.max_new = p.max_new;
    a.cap = p.c.width * p.c.page;
    a.few = few;
    a.withheld = p.withheld;
    a.scale_log2 = p.scale_log2;
    const bool d128 = p.d == 128;
    const void* fn = d128 ? reinterpret_cast<const void*>(paged_items_kernel<128>) : reinterpret_cast<const void*>(paged_items_kernel<64>);
    const int smem = d128 ? PwShape<128>::SMEM : PwShape<64>::SMEM;
    void* args[] = {&a};
    cudaError_t e = launch_pdl(d128 ? reinterpret_cast<const void*>(paged_terms_kernel<128>) : reinterpret_cast<const void*>(paged_terms_kernel<64>), args,
                               (int)((rows * (p.d / 16) + 255) / 256), 0, s, 256);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e == cudaSuccess) e = launch_pdl(fn, args, kSMs, smem, s, kPwThreads);
    if (e != cudaSuccess) return e;
    int slices = 32;
    void* jargs[] = {&a, &slices};
    return launch_pdl(d128 ? reinterpret_cast<const void*>(paged_join_kernel<128>) : reinterpret_cast<const void*>(paged_join_kernel<64>), jargs,
                      kSMs * slices, 0, s, 128);
}

}  // namespace tpk
