// Attention of a packed batch over the shards' KV caches, with an optional
// prefix that the batch shares.
//
//   o = sum_j w_j v_j / sum_j w_j,  w_j = 2^(s_j - m),  s_j = q . k_j log2(e) / sqrt(d)
//
// (0 / 0 where every s_j is -inf: such a row is NaN, and zeros are written only
// to rows whose position lies outside the cache) in one pass over the keys with
// a running m and sum, in up to four launches:
//   attn_plan_kernel     one CTA turns the offsets and lengths into a list of
//                        items, longest first, and cuts long items into parts
//                        where the batch has too few of them for the machine
//                        (a call of very few rows does without it);
//   attn_items_kernel    persistent, one CTA per SM: items of many query rows;
//   attn_narrow_kernel   the same for items of few query rows;
//   attn_combine_kernel  joins the parts of a row.
// A call whose sequences bring few tokens each treats a shared prefix as items
// of its own, whose rows are the batch's tokens whatever their sequence: its
// keys are read once for the batch. Otherwise the prefix's blocks precede the
// sequence's own in the item's list of key blocks.
#include <climits>
#include <cstring>
#include <mutex>

#include <cuda.h>
#include <cudaTypedefs.h>

#include "attn.cuh"
#include "common.cuh"
#include "stream.cuh"
#include "tcgen05.cuh"
#include "tp_internal.h"

namespace tpk {

constexpr int kAtM = 128;               // query rows per tile: 128 / G tokens of the G heads of a KV head
constexpr int kAtK = 128;               // keys per block
constexpr int kAtBuckets = 512;         // item lengths told apart when sorting
constexpr int kAtMinPart = 2;           // blocks of the shortest part of a narrow item worth its join
constexpr int kAtMinCut = 4;            // ... and of a wide one, which has more rows to join
constexpr int kAtMaxParts = 16;
constexpr int kAtNarrow = 32;           // rows of an item at most that the narrow kernel can take

enum AttnKind : int { AT_PREFIX = 1, AT_OWN = 2 };   // key blocks of an item: the prefix's, the sequence's own

// blocks of a sequence's own cache that a tile ending at position `end` (exclusive) needs
__device__ __forceinline__ int own_blocks(int64_t end, int max_kv) {
    const int64_t e = end < 0 ? 0 : (end > max_kv ? max_kv : end);
    return (int)((e + kAtK - 1) / kAtK);
}

// Splits `nb` blocks into parts of about `target` blocks each: equal ones when nb exceeds it by half, or, where `rest` is
// set, parts of `target` and a shorter last one, of at least kAtMinCut blocks.
__device__ __forceinline__ void part_split(int nb, int target, bool rest, int& parts, int& len) {
    parts = 1;
    len = nb;
    if (rest) {
        parts = max(1, (int)((unsigned)(nb - kAtMinCut + target) / (unsigned)target));
        len = parts > 1 ? max(target, (int)((unsigned)(nb + parts - 1) / (unsigned)parts)) : nb;
    } else if (nb > target + target / 2) {
        parts = (unsigned)(nb + target - 1) / (unsigned)target;
        len = (unsigned)(nb + parts - 1) / (unsigned)parts;
        parts = (unsigned)(nb + len - 1) / (unsigned)len;
    }
}

// One CTA. Three passes over the tiles: check and sum up, count the items of
// each length, place them. A lane takes a sequence (the first of them stay in
// its registers), a warp the tiles of a long sequence together. The items are
// sorted by length; CTAs take them from the front.
//
// An item is cut into parts, which are joined at the end, where whole items
// would leave SMs without work: all long ones, when there are fewer than SMs; one
// that is longer than an even share of all; and those of a last round that has
// few (two rounds of equal items for 160 on 152 SMs end almost twice as late as
// one). Parts cost their partial results' way to memory and back.
//
// Integer atomics place the items of a length and the rows of partial results:
// their order decides who does an item when and where a partial lies, not what
// is added to what. Which of several items of a length belong to the last round
// must not depend on it, since a cut item is summed up in another order: those
// are ranked by warp and, within one, in the order in which it comes to them.
//
// Bound by latency, 3 to 5 us of it: instructions that run once come from
// memory, and what every warp computes for itself takes its turn. So the three
// passes are one loop, their tiles come from one place, and the warps are eight
// (32 warps and the passes written out: decode of 64 behind 4096 rows 59 us, of
// 256 behind 16384 rows 220; now 53 and 207. 16 warps: 55 and 208).
constexpr int kPlanThreads = 256, kPlanWarps = kPlanThreads / 32;
static_assert(2 * kAtBuckets == 4 * kPlanThreads, "four buckets per thread");

// an even share of the blocks of all KV heads, rounded up (2^-21 for the roundings of the product and the quotient)
__device__ __forceinline__ int even_share(unsigned long long blocks, int heads, float parts) {
    const float q = (float)blocks * (float)heads * (1.f / parts) * (1.f + 0x1p-21f) + 1.f;
    return max(kAtMinPart, (int)fminf(q, 0x1p29f));
}
// narrow items: two parts per half of a CTA (time goes by the bytes: parts cost little)
__device__ __forceinline__ int narrow_share(unsigned long long blocks, int heads) { return even_share(blocks, heads, 4.f * kSMs); }

__device__ __forceinline__ int warp_scan(int x, int lane) {          // inclusive
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += v;
    }
    return x;
}
// the lane whose range [before, before + its number) holds i, before ascending
__device__ __forceinline__ int warp_owner(int before, int i) {
    int at = 0;
    for (int o = 16; o; o >>= 1)
        if (__shfl_sync(0xffffffffu, before, at + o) <= i) at += o;
    return at;
}

__global__ void __launch_bounds__(kPlanThreads) attn_plan_kernel(const RaggedAttnParams p) {
    __shared__ __align__(16) int s_hist[2 * kAtBuckets];             // wide items, narrow items
    __shared__ unsigned long long s_blocks[2][kPlanWarps];           // per warp: blocks of wide and narrow tiles
    __shared__ int s_tiles[kPlanWarps], s_longest[kPlanWarps];       // wide tiles
    __shared__ int s_few[kPlanWarps], s_few_longest[kPlanWarps];     // narrow tiles
    __shared__ int s_warp[kPlanWarps];
    __shared__ __align__(16) int s_ties[kPlanWarps * kAtBuckets];    // per warp: wide items of each length
    __shared__ int s_rows, s_chunks, s_edge, s_edge_at;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    constexpr unsigned kAll = 0xffffffffu;
    pdl_trigger();
    reinterpret_cast<int4*>(s_hist)[tid] = make_int4(0, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < kPlanWarps * kAtBuckets / 4; i += kPlanThreads) reinterpret_cast<int4*>(s_ties)[i + tid] = make_int4(0, 0, 0, 0);
    const int G = (unsigned)p.hq_s / (unsigned)p.hkv_s, per = 2 * ((unsigned)kAtM / (unsigned)G);      // tokens per item
    const int heads = p.N * p.hkv_s;
    if (tid == 0) {
        s_rows = 2 * p.T * heads * G;                                // behind the places of part 0
        s_chunks = 0;
        s_edge = s_edge_at = 0;
    }
    const int n_prefix = (p.prefix_len + kAtK - 1) / kAtK;           // prefix blocks
    const int in_item = p.shared ? 0 : n_prefix;
    const int lanes = min(32, (p.B + kPlanWarps - 1) / kPlanWarps);  // sequences per warp and round
    pdl_wait();

    int bad = 0, out = 0;
    const int n_tok = p.cu[p.B];
    auto load = [&](int b0, int& c, int& n, int& pos) {
        const int b = b0 + lane;
        c = n = pos = 0;
        if (lane < lanes && b < p.B) {
            c = p.cu[b];
            const int c1 = p.cu[b + 1];
            pos = p.pos[b];
            if (c1 < c || c < 0 || c1 > p.T || (b == 0 && c != 0)) bad = 1;
            else if (c1 > c && (pos < 0 || (int64_t)pos + (c1 - c) > p.max_kv)) out = 1;
            if (!bad) n = c1 - c;
        }
    };
    int c0, n0, q0;                                                  // the lane's sequence of the first round
    load(warp * lanes, c0, n0, q0);

    unsigned long long wide_blocks = 0, narrow_blocks = 0;
    int wide_tiles = 0, longest = 0, few_tiles = 0, few_longest = 0;
    int narrow = p.narrow;                                           // most rows of a narrow item
    int target_w = 0, target_n = 0;                                  // the longest parts
    bool rests = false;                                              // wide items: of that length but the last
    int last_from = INT_MAX, last_parts = 1;                         // a last round's items and their parts
    int edge = -1, edge_at = 0;                                      // the bucket in which it begins, the warp's next place there
    int n_wide = 0, n_items = 0;
    const int own = p.shared ? AT_OWN : AT_OWN | AT_PREFIX;

#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
        // The warp's tiles, 32 at a time: those of a round of its sequences back to back, then its share of a shared prefix's.
        int next = warp * lanes, c = c0, n = n0, q = q0;             // the lane's sequence of the round
        int b0 = 0, before = 0, total = 0, i0 = 0, step = 32;
        bool shared = pass && p.shared;
        int kind = own;
#pragma unroll 1
        while (true) {
            if (i0 >= total) {
                if (next < p.B) {
                    if (next != warp * lanes) load(next, c, n, q);
                    const int tiles = (unsigned)(n + per - 1) / (unsigned)per;
                    before = warp_scan(tiles, lane);
                    total = __shfl_sync(kAll, before, 31);
                    before -= tiles;
                    b0 = next;
                    i0 = 0;
                    next += kPlanWarps * lanes;
                } else if (shared) {                                 // as one sequence of all tokens
                    shared = false;
                    kind = AT_PREFIX;
                    c = q = b0 = 0;
                    n = n_tok;
                    before = lane ? INT_MAX : 0;
                    total = (unsigned)(n_tok + per - 1) / (unsigned)per;
                    i0 = 32 * warp;
                    step = 32 * kPlanWarps;
                } else {
                    break;
                }
                continue;
            }
            const int tile = i0 + lane, owner = warp_owner(before, tile);
            const int at = (tile - __shfl_sync(kAll, before, owner)) * per;
            const int b = b0 + owner, t0 = __shfl_sync(kAll, c, owner) + at;
            const int qpos = (int)((int64_t)__shfl_sync(kAll, q, owner) + at);
            const int left = __shfl_sync(kAll, n, owner) - at, k = tile < total ? min(per, left) : 0;     // tokens
            i0 += step;
            const bool live = k > 0, nar = k * G <= narrow;
            const int nb = kind == AT_PREFIX ? n_prefix : in_item + own_blocks((int64_t)qpos + k, p.max_kv);
            if (pass == 0) {
                if (live && nar) {
                    narrow_blocks += nb;
                    ++few_tiles;
                    few_longest = max(few_longest, nb);
                }
                if (live && !nar) {
                    wide_blocks += nb;
                    ++wide_tiles;
                    longest = max(longest, nb);
                }
                continue;
            }
            int parts, len;
            part_split(nb, nar ? target_n : target_w, rests && !nar, parts, len);
            int* rest = &s_hist[(nar ? 2 : 1) * kAtBuckets - 1 - min(nb - (parts - 1) * len, kAtBuckets - 1)];
            int* full = &s_hist[(nar ? 2 : 1) * kAtBuckets - 1 - min(len, kAtBuckets - 1)];
            int e0 = 0, e1 = 0;                                      // places of the parts but the last, and of the last
            if (live) {
                if (parts > 1) e0 = atomicAdd(full, parts - 1);
                e1 = atomicAdd(rest, 1);
            }
            if (pass == 1) {                                         // (nothing else is cut where a last round is)
                if (last_parts > 1 && live && !nar) atomicAdd(&s_ties[warp * kAtBuckets + (int)(rest - s_hist)], 1);
                continue;
            }
            if (edge >= 0) {
                const unsigned tied = __ballot_sync(kAll, live && !nar && rest - s_hist == edge);
                if (tied >> lane & 1) e1 = edge_at + __popc(tied & ((1u << lane) - 1u));
                edge_at += __popc(tied);
            }

            int entries = live ? parts : 0;
            if (live && parts == 1 && !nar && e1 >= last_from) {
                e0 = last_from + (e1 - last_from) * last_parts;
                parts = max(1, min(last_parts, nb / kAtMinPart));
                len = (nb + parts - 1) / parts;
                parts = max(1, (nb + len - 1) / max(len, 1));
                e1 = e0 + parts - 1;
                entries = last_parts;                                // those behind the parts: no rows
            }
            // partial results: part 0 of a tile at the place of its tokens, the others where there is room
            const int rows = heads * k * G;
            int row0 = -1, row1 = 0, chunks = 0;
            if (live && (parts > 1 || p.shared)) {
                row0 = heads * G * ((kind & AT_OWN ? 0 : p.T) + t0);
                if (parts > 1) row1 = atomicAdd(&s_rows, (parts - 1) * rows);
                if (kind & AT_OWN) chunks = (k * G + 7) / 8;
                else p.prefix_groups[(unsigned)t0 / (unsigned)per] = make_int2(row1, parts);
            }
            const int upto = warp_scan(chunks, lane), sum = __shfl_sync(kAll, upto, 31);
            if (sum) {
                int to = 0;
                if (lane == 0) to = atomicAdd(&s_chunks, sum);
                to = __shfl_sync(kAll, to, 0) + upto - chunks;
#pragma unroll 1
                for (int j = 0; j < chunks; ++j) p.chunks[to + j] = AttnChunk{t0, k, qpos, row1, parts, j, 0, 0};
            }
#pragma unroll 1
            for (int j = 0; j < entries; ++j) {
                const int row = j && row0 >= 0 ? row1 + (j - 1) * rows : row0;
                AttnItem x = {t0, k, b, qpos, j * len, min(nb, (j + 1) * len), kind, row};
                if (j >= parts) x = AttnItem{0, 0, 0, 0, 0, 0, kind, -1};
                p.items[j == parts - 1 ? e1 : e0 + j] = x;
            }
        }

        if (pass == 0) {
            // ---- the sums over the warps; the longest parts
            for (int o = 16; o; o >>= 1) {
                wide_blocks += __shfl_xor_sync(kAll, wide_blocks, o);
                narrow_blocks += __shfl_xor_sync(kAll, narrow_blocks, o);
            }
            wide_tiles = __reduce_add_sync(kAll, wide_tiles);
            longest = __reduce_max_sync(kAll, longest);
            few_tiles = __reduce_add_sync(kAll, few_tiles);
            few_longest = __reduce_max_sync(kAll, few_longest);
            if (lane == 0) {
                s_few[warp] = few_tiles;
                s_few_longest[warp] = few_longest;
                s_tiles[warp] = wide_tiles;
                s_longest[warp] = longest;
                s_blocks[0][warp] = wide_blocks;
                s_blocks[1][warp] = narrow_blocks;
            }
            if (__syncthreads_or(bad)) {
                if (tid < (int)(sizeof(AttnCtl) / sizeof(int))) reinterpret_cast<int*>(p.ctl)[tid] = 0;
                if (tid == 0) set_status(p.status, TP_ERR_SHAPE);
                return;
            }
            if (out) set_status(p.status, TP_ERR_CAPACITY);
            constexpr int kMask = kPlanWarps - 1;
            wide_blocks = s_blocks[0][lane & kMask];
            narrow_blocks = s_blocks[1][lane & kMask];
            for (int o = kPlanWarps / 2; o; o >>= 1) {
                wide_blocks += __shfl_xor_sync(kAll, wide_blocks, o);
                narrow_blocks += __shfl_xor_sync(kAll, narrow_blocks, o);
            }
            wide_tiles = __reduce_add_sync(kAll, lane < kPlanWarps ? s_tiles[lane & kMask] : 0);
            longest = __reduce_max_sync(kAll, s_longest[lane & kMask]);
            few_tiles = __reduce_add_sync(kAll, lane < kPlanWarps ? s_few[lane & kMask] : 0);
            // A few narrow items beside many wide ones are done as such: their own kernel gets an SM only when the wide one
            // leaves it, and its chain of an item's blocks then follows. Tiles of one prompt and of single tokens over 2000
            // keys, 8 KV heads, apart and together: 32 and 4 52 and 48 us, 64 and 16 132 and 125, 64 and 32 153 and 152, 64
            // and 64 187 and 193. Not where the wide ones hardly fill the SMs once: 20 and 5 58 and 60, 8 and 2 28 and 37.
            if (few_tiles <= wide_tiles / 4 && wide_tiles * (int64_t)heads >= kSMs + kSMs / 2) {
                narrow = 0;
                wide_tiles += few_tiles;
                wide_blocks += narrow_blocks;
                narrow_blocks = 0;
                longest = max(longest, __reduce_max_sync(kAll, s_few_longest[lane & kMask]));
            }
            if (p.shared) {
                const int tiles = (unsigned)(n_tok + per - 1) / (unsigned)per;
                const int small = tiles && (n_tok - (tiles - 1) * per) * G <= narrow;
                wide_tiles += tiles - small;
                wide_blocks += (unsigned long long)(tiles - small) * n_prefix;
                if (small) narrow_blocks += n_prefix;
                if (tiles > small) longest = max(longest, n_prefix);
            }
            const long long items = (long long)wide_tiles * heads;
            target_n = narrow_share(narrow_blocks, heads);
            target_w = max(kAtMinCut, even_share(wide_blocks, heads, kSMs));
            if (items && items <= kSMs) {
                // The parts per item that are done first, in microseconds, k of them in lane k - 1: rounds of parts, each two
                // blocks' time longer than its blocks and the first seven more (half as long again beside narrow items,
                // which keep the memory busy); what the SMs that are left do not read of the narrow items meanwhile; and
                // the joining, 4.4 MB of float32 results a microsecond there and back. Both sides, 8 KV heads: 256 tokens
                // behind 16384, k = 1/2/3/4/6: 252/209/225/238/248 us; 64 behind 4096, k = 1/2/3/4/6/8: 93/73/65/62/56/58
                // us; a chunk of 512 behind 30001, k = 1/2/3/4/6/8: 331/195/249/202/210/217 us.
                // Lanes 16 and up take k parts of one length on an SM each and a shorter last one for the SMs that are left,
                // which do one after the other: the chunk in two equal parts uses 128 SMs and takes 188 us, in two and a
                // rest 176; one of 1024 331 and 321, of 256 107 and 101.
                const int all = (int)items, k = (lane & 15) + 1;
                int len = (unsigned)(longest + k - 1) / (unsigned)k, sms = min(k * all, kSMs), time = len, parts = k;
                bool ok = k == 1 || (k * all <= 3 * kSMs && len >= kAtMinCut);
                if (lane & 16) {
                    const int turns = (unsigned)(all + kSMs - k * all - 1) / (unsigned)max(kSMs - k * all, 1);
                    len = (unsigned)(turns * (longest + 4)) / (unsigned)(turns * k + 1) + 1;
                    ok = k * all < kSMs && longest - k * len >= kAtMinCut;
                    sms = kSMs;
                    parts = k + 1;
                    time = len;
                } else {
                    time = (k * all + kSMs - 1) / kSMs * (len + 2) - 2;
                }
                const float bytes = (float)narrow_blocks * heads * (kAtK * 4) * p.d;
                const float wide_us = (float)(time + 9) * (narrow_blocks ? 1.6f : 1.1f);
                const float left = fmaxf(0.f, bytes - wide_us * fminf(6.5e6f, (kSMs - sms) * 6e4f));
                const float join = (float)(all * 2 * kAtM) * p.d * 8 / 4.4e6f;
                const float t = ok ? wide_us + left / 6.5e6f + (parts > 1 ? parts * join : 0.f) : INFINITY;
                const unsigned best = __reduce_min_sync(kAll, __float_as_uint(t));       // positive: ordered as their bits
                const int lane_of = __ffs(__ballot_sync(kAll, __float_as_uint(t) == best)) - 1;
                target_w = __shfl_sync(kAll, len, lane_of);
                rests = lane_of & 16;
            }
            // a last round of few items, if nothing else is cut: parts for its items
            const int rounds = items <= 3 * kSMs ? (int)items / kSMs : 0;
            if (rounds && !rests && longest <= target_w + target_w / 2) {
                last_from = (unsigned)(rounds * kSMs + heads - 1) / (unsigned)heads;
                const int rest = wide_tiles - last_from;
                last_parts = rest > 0 ? min(kAtMaxParts, (int)((unsigned)kSMs / (unsigned)(rest * heads))) : 1;
                if (last_parts < 2) last_from = INT_MAX, last_parts = 1;
            }
        } else if (pass == 1) {
            // ---- where the items of each length begin: exclusive sums over the buckets, four per thread
            __syncthreads();
            const int4 x = reinterpret_cast<const int4*>(s_hist)[tid];
            const int mine = x.x + x.y + x.z + x.w, incl = warp_scan(mine, lane);
            if (lane == 31) s_warp[warp] = incl;
            __syncthreads();
            const int of_warp = s_warp[lane & (kPlanWarps - 1)];
            const int sorted = __reduce_add_sync(kAll, lane < kPlanWarps / 2 ? of_warp : 0);           // wide items
            const int more = last_parts > 1 ? (sorted - last_from) * (last_parts - 1) : 0;      // the last round's parts
            n_wide = sorted + more;
            n_items = __reduce_add_sync(kAll, lane < kPlanWarps ? of_warp : 0) + more;
            int e = __reduce_add_sync(kAll, lane < warp ? of_warp : 0) + incl - mine + (warp >= kPlanWarps / 2 ? more : 0);
            const int4 begin = make_int4(e, e + x.x, e + x.x + x.y, e + x.x + x.y + x.z);
            reinterpret_cast<int4*>(s_hist)[tid] = begin;
            if (warp < kPlanWarps / 2 && e <= last_from && last_from < e + mine) {
                const int i = (last_from >= begin.y) + (last_from >= begin.z) + (last_from >= begin.w);
                s_edge = 4 * tid + i;
                s_edge_at = i == 0 ? begin.x : i == 1 ? begin.y : i == 2 ? begin.z : begin.w;
            }
            __syncthreads();
            if (last_parts > 1) {
                edge = s_edge;
                edge_at = s_edge_at + __reduce_add_sync(kAll, lane < warp ? s_ties[lane * kAtBuckets + edge] : 0);
            }
        }
    }
    __syncthreads();
    if (tid == 0) {
        AttnCtl c = {};
        c.n_tokens = n_tok;
        c.n_wide = n_wide;
        c.n_items = n_items;
        c.n_chunks = s_chunks;
        *p.ctl = c;
    }
}

// ---------------------------------------------------------------------------
// The items on the tensor cores. An item is two tiles of 128 query rows (the
// G heads of a KV head for 128 / G consecutive tokens each) over a range of
// key blocks; both tiles use every block that is loaded.
//   warp 0        TMA: the Q tiles, then K and V blocks of 128 keys, in the
//                 order in which they are used, into a ring of slots;
//   warps 1, 2    the products of tile 0 and 1 in tensor memory (S_0, S_1, O_0,
//                 O_1): S_t = Q_t K^T; O_t += P_t V with P_t read from tensor
//                 memory (bf16, over S_t), in halves as the softmax writes it.
//                 While one tile's softmax runs, the other's products do, and
//                 the next item's S_t is issued behind this item's last O_t;
//   warps 4-7,    softmax of tile 0 and 1, one row per thread: masked maximum,
//   8-11          P = 2^(S - m) rounded to bf16 (its sum is taken before), m
//                 moving only when a row's maximum grows by more than 2^8
//                 (O is then rescaled; a weight of 2^8 is as exact in bf16 and
//                 float32 as one of 1);
//   warp 3        V blocks that some row of the item does not see to their end
//                 are made finite before their product (0 * inf is not 0);
//   warps 12-15   the results O / l (or O, m and l of a part) are written while
//                 the next item is under way.
// The items' ranges of blocks are walked in the same order by every role; all
// waits are bounded.
//
// P is held in bf16 because a product's operands are of one type and V is bf16:
// float32 weights would need V widened in shared memory and products of tf32, at
// half the rate that bounds the kernel. A weight is off by at most 2^-8 of
// itself, with either sign; over the listed calls the results are 0.0019 to
// 0.0023 of their norm off, and 0.0016 to 0.0017, which is their own rounding to
// bf16, with float32 weights. Sums, maxima and O stay float32.
//
// Bound by the tensor cores: 256 rows x 128 keys are 2048 cycles of products for
// d = 128 (2053 measured, products alone). Causal prompts of 32 heads: 8192
// tokens 342 us, 1.61 PFLOP/s, 16384 tokens 1350 to 1380 us, 1.6 PFLOP/s of 1.88
// measured for a library product; the block takes about 2500 cycles, and the
// power limit takes its share of the clock. For d = 64 the products take 1024
// cycles and the 32768 exponentials, at 4 cycles for 32 of a quarter of the SM,
// as long, but 8192 tokens take 290 us, 0.95 PFLOP/s: the chain of maximum,
// exponentials and hand-over bounds it, with each unit at half its rate. For
// short prompts an item's beginning and end count: the first 10 to 14 us with
// cold code, each later one 3 to 6 (16 prompts behind 2048 keys: 56 us for 15 us
// of products).
//
// Taken against (8192 tokens): the scores read twice, once for the maximum, once
// for the weights, so that they need no registers: 400 for 357 us; the products
// of both tiles without turns: 479 for 359; spilled registers or longer loops
// cost more than any of their instructions, which the split of registers and the
// waits out of line come from.
// ---------------------------------------------------------------------------

constexpr int kAtThreads = 512;
constexpr int kAtQueue = 4;               // items read ahead
constexpr float kAtRescale = 8.0f;
constexpr int kAtRegsIo = 88, kAtRegsSoftmax = 160, kAtRegsOut = 104;
static_assert(kAtRegsIo + 2 * kAtRegsSoftmax + kAtRegsOut <= 4 * 128, "the launch's registers");

template <int D>
struct AtShape {
    static constexpr int NKB = D / 64;
    static constexpr int QB = kAtM * D * 2;             // one Q tile
    static constexpr int KB = kAtK * D * 2;             // one K or V block
    static constexpr int RING = D == 128 ? 5 : 10;
    static constexpr int HEAD = 1024;                   // barriers
    static constexpr int STAT = 2 * kAtM * 8;           // (m, l) of the tiles' rows
    static constexpr int SMEM = HEAD + 2 * QB + RING * KB + STAT;
};

struct AtArgs {
    CUtensorMap tq;                       // q as [N T][hq_s][D], boxes of 128 / G tokens x G heads x 64
    CUtensorMap tqn;                      // the same with boxes of kAtNarrow / G tokens
    CUtensorMap tk[TP_MAX_SHARDS];        // caches as [max_batch hkv_s][max_kv][D], boxes of 128 (narrow: kAnBox) rows x 64
    CUtensorMap tv[TP_MAX_SHARDS];
    CUtensorMap pk[TP_MAX_SHARDS];        // prefix as [hkv_s][prefix_len][D] (rows past it read as zeros)
    CUtensorMap pv[TP_MAX_SHARDS];
    const bf16* v[TP_MAX_SHARDS];
    bf16* out;                            // [N][T][hq_s][D]
    float* part_o;                        // [rows][D]
    float2* part_ml;                      // [rows] (m, l)
    const AttnItem* items;
    AttnCtl* ctl;
    int after_wide;                       // narrow kernel: the wide one is launched before it
    int few;                              // narrow kernel: no plan kernel ran
    int B;                                // (few) as below to prefix_groups
    const int* cu;
    const int* pos;
    AttnChunk* chunks;
    int2* prefix_groups;
    int N, T, hq_s, hkv_s, G, tpt, max_kv, prefix_len;
    float scale_log2;
    int* status;
};

// One item for one KV head of one shard. nb0, nb1: key blocks of its tiles.
struct __align__(16) AtWork {
    int r, kvh, h;                        // shard, KV head of the shard, KV head of all
    int t0, ntok, b, qpos, blk0, part;
    int nP, nt, nb0, nb1, nb;             // prefix blocks in the list, tiles, blocks of the tiles and of both
    int end, reserved;                    // 1: there are no more items
};
static_assert(sizeof(AtWork) == 64, "four 16-byte words of the queue");

__device__ __forceinline__ void at_fill(const AtArgs& a, const int4& x, const int4& y, int h, AtWork& w) {
    w.h = h;
    w.r = h / a.hkv_s;
    w.kvh = h - w.r * a.hkv_s;
    w.t0 = x.x;
    w.ntok = x.y;
    w.b = x.z;
    w.qpos = x.w;
    w.blk0 = y.x;
    const int blk1 = y.y, kind = y.z;
    w.part = y.w;
    w.nP = (kind & AT_PREFIX) ? (a.prefix_len + kAtK - 1) / kAtK : 0;
    w.nt = w.ntok > a.tpt ? 2 : 1;
    const int n0 = min(w.ntok, a.tpt);
    const int e0 = w.nP + ((kind & AT_OWN) ? own_blocks((int64_t)w.qpos + n0, a.max_kv) : 0);
    const int e1 = w.nP + ((kind & AT_OWN) ? own_blocks((int64_t)w.qpos + w.ntok, a.max_kv) : 0);
    w.nb0 = max(0, min(blk1, e0) - w.blk0);
    w.nb1 = w.nt > 1 ? max(0, min(blk1, e1) - w.blk0) : 0;
    w.nb = max(w.nb0, w.nb1);
    w.end = w.reserved = 0;
}
__device__ __forceinline__ void at_load(const AtArgs& a, int e, int4& x, int4& y) {
    x = __ldcg(reinterpret_cast<const int4*>(a.items + e));
    y = __ldcg(reinterpret_cast<const int4*>(a.items + e) + 1);
}
__device__ __forceinline__ void at_decode(const AtArgs& a, int e, int h, AtWork& w) {
    int4 x, y;
    at_load(a, e, x, y);
    at_fill(a, x, y, h, w);
}

// Block j of an item: its first key in the prefix (own = false) or in the sequence's own cache.
__device__ __forceinline__ int at_block(const AtWork& w, int j, bool& own) {
    const int k = w.blk0 + j;
    own = k >= w.nP;
    return (own ? k - w.nP : k) * kAtK;
}
// end of an item's own keys
__device__ __forceinline__ int at_kend(const AtArgs& a, const AtWork& w) {
    const int64_t e = (int64_t)w.qpos + w.ntok;
    return (int)(e < 0 ? 0 : (e > a.max_kv ? a.max_kv : e));
}
// whether the V block at own key `key0` has rows that some row of the item does not see
__device__ __forceinline__ bool at_ragged(const AtWork& w, int key0) { return (int64_t)key0 + kAtK > (int64_t)w.qpos + 1; }

// Whether a bf16 of the word is infinite or NaN: adding one to a full exponent carries out of it.
__device__ __forceinline__ uint32_t not_finite(uint32_t x) { return ((x & 0x7F807F80u) + 0x00800080u) & 0x80008000u; }
__device__ __forceinline__ uint32_t only_finite(uint32_t x) {
    if ((x & 0x7F80u) == 0x7F80u) x &= 0xFFFF0000u;
    if ((x & 0x7F800000u) == 0x7F800000u) x &= 0xFFFFu;
    return x;
}

// One warp: rows 0 .. valid - 1 of a V block without infinities and NaN, the
// rows behind them zeros as far as a product of 16 keys reads. Whether the lane
// found one. A step is four rows of 128 bytes; the swizzle moves 16-byte units
// within a row only. The common block is only looked at: x * 0 summed up is NaN
// if any x is not finite, one instruction for two values.
template <int D>
__device__ __forceinline__ int v_block_finite(unsigned char* block, int lane, int valid) {
    const int rows = (valid + 15) & ~15;
    uint32_t sum[4] = {0, 0, 0, 0};
    auto look = [&](uint32_t& s, uint32_t x) { asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(s) : "r"(x), "r"(0u)); };
#pragma unroll
    for (int c = 0; c < D / 64; ++c) {
        uint4* base = reinterpret_cast<uint4*>(block + c * (kAtK * 128)) + lane;
#pragma unroll 1
        for (int r0 = 0; r0 < rows; r0 += 16) {
            uint4 x[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = base[(r0 / 4 + i) * 32];
            if (r0 + 16 > valid) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (r0 + 4 * i + (lane >> 3) >= valid) x[i] = base[(r0 / 4 + i) * 32] = make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                look(sum[0], x[i].x);
                look(sum[1], x[i].y);
                look(sum[2], x[i].z);
                look(sum[3], x[i].w);
            }
        }
    }
    if (!__any_sync(0xffffffffu, not_finite(sum[0]) | not_finite(sum[1]) | not_finite(sum[2]) | not_finite(sum[3]))) return 0;
    int found = 0;
#pragma unroll 1
    for (int c = 0; c < D / 64; ++c)
#pragma unroll 1
        for (int i = 0; i < rows / 4; ++i) {
            uint4* q = reinterpret_cast<uint4*>(block + c * (kAtK * 128)) + lane + i * 32;
            const uint4 x = *q;
            if (not_finite(x.x) | not_finite(x.y) | not_finite(x.z) | not_finite(x.w)) {
                *q = make_uint4(only_finite(x.x), only_finite(x.y), only_finite(x.z), only_finite(x.w));
                found = 1;
            }
        }
    return found;
}

// Row `m` of a V block: zeros where it lies behind the last key, and no
// infinities or NaN. Whether it held one.
template <int D>
__device__ __forceinline__ int v_row_finite(unsigned char* block, int m, bool past) {
    int found = 0;
#pragma unroll
    for (int c = 0; c < D / 64; ++c)
#pragma unroll 1
        for (int u = 0; u < 8; ++u) {
            uint4* q = reinterpret_cast<uint4*>(block + m * 128 + c * (kAtK * 128) + ((u ^ (m & 7)) << 4));
            if (past) {
                *q = make_uint4(0, 0, 0, 0);
                continue;
            }
            uint4 x = *q;
            uint32_t* y = reinterpret_cast<uint32_t*>(&x);
            if (not_finite(y[0]) | not_finite(y[1]) | not_finite(y[2]) | not_finite(y[3])) {
                *q = make_uint4(only_finite(y[0]), only_finite(y[1]), only_finite(y[2]), only_finite(y[3]));
                found = 1;
            }
        }
    return found;
}

template <int D>
__global__ void __launch_bounds__(kAtThreads, 1) attn_items_kernel(const __grid_constant__ AtArgs a) {
    using Sh = AtShape<D>;
    constexpr int R = Sh::RING;
    extern __shared__ __align__(1024) unsigned char smem[];
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem);
    uint64_t* q_full = bars;              // [2] per tile
    uint64_t* q_empty = q_full + 2;       // [2]
    uint64_t* s_full = q_empty + 2;       // [2]
    uint64_t* p_half = s_full + 2;        // [2] P of the first 64 keys
    uint64_t* p_full = p_half + 2;        // [2]
    uint64_t* o_full = p_full + 2;        // [2] an item's last product of the tile
    uint64_t* o_empty = o_full + 2;       // [2] O has been read
    uint64_t* st_full = o_empty + 2;      // [2] (m, l)
    uint64_t* st_empty = st_full + 2;     // [2]
    uint64_t* kv_full = st_empty + 2;     // [R]
    uint64_t* kv_empty = kv_full + R;     // [R]
    uint64_t* v_clean = kv_empty + R;     // [R] the slot's ragged V block is finite
    uint64_t* note = v_clean + R;         // [kAtQueue] the item's notes are written
    uint64_t* turn = note + kAtQueue;     // [2] whose products are next
    uint64_t* item_full = turn + 2;       // [kAtQueue]
    uint64_t* item_empty = item_full + kAtQueue;
    uint64_t* done = item_empty + kAtQueue;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    volatile int* s_poison = reinterpret_cast<volatile int*>(tmem_slot + 2);   // [kAtQueue] an item's V had infinities or NaN
    AtWork* queue = reinterpret_cast<AtWork*>(smem + Sh::HEAD - kAtQueue * sizeof(AtWork));
    static_assert((18 + 3 * R + 2 + 3 * kAtQueue + 1) * 8 + 8 + 4 * kAtQueue <= Sh::HEAD - kAtQueue * sizeof(AtWork), "the head's words");
    unsigned char* sq = smem + Sh::HEAD;
    unsigned char* ring = sq + 2 * Sh::QB;
    float2* stat = reinterpret_cast<float2*>(ring + R * Sh::KB);     // [2][kAtM]

    const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&q_full[i], 1);
            mbar_init(&q_empty[i], 1);
            mbar_init(&s_full[i], 1);
            mbar_init(&p_half[i], 4);
            mbar_init(&p_full[i], 4);
            mbar_init(&o_full[i], 1);
            mbar_init(&o_empty[i], 4);
            mbar_init(&st_full[i], 4);
            mbar_init(&st_empty[i], 4);
        }
        for (int i = 0; i < R; ++i) {
            mbar_init(&kv_full[i], 1);
            mbar_init(&kv_empty[i], 3);
            mbar_init(&v_clean[i], 1);
        }
        mbar_init(&turn[0], 1);
        mbar_init(&turn[1], 1);
        for (int i = 0; i < kAtQueue; ++i) {
            mbar_init(&item_full[i], 1);
            mbar_init(&item_empty[i], 15);
            mbar_init(&note[i], 1);
        }
        mbar_init(done, 2);
        *abort_flag = (smem_u32(sq) & 1023u) ? 1 : 0;
        if (*abort_flag) set_status(a.status, TP_ERR_ALIGN);
        fence_mbar_init();
    }
    if (warp == 1) tmem_alloc(smem_u32(tmem_slot), 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = uniform(*tmem_slot);
    pdl_wait();
    pdl_trigger();                        // only now: the narrow kernel relies on the lists being there when it starts
    // The copying thread reads the list ahead of the other roles and leaves the items in a queue in shared memory; this
    // gives the k-th of them to a warp.
    auto item_done = [&](int k) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&item_empty[k % kAtQueue]);
    };
    auto item = [&](int k, AtWork& w, bool hold = false) {  // hold: the warp calls item_done itself
        const int q = k % kAtQueue;
        if (!__all_sync(0xffffffffu, mbar_wait(&item_full[q], (k / kAtQueue) & 1, abort_flag, a.status))) return false;
        const int4* x = reinterpret_cast<const int4*>(&queue[q]);
        const int4 x0 = x[0], x1 = x[1], x2 = x[2], x3 = x[3];
        if (!hold) item_done(k);
        w.r = x0.x, w.kvh = x0.y, w.h = x0.z, w.t0 = x0.w;
        w.ntok = uniform(x1.x), w.b = x1.y, w.qpos = uniform(x1.z), w.blk0 = uniform(x1.w);
        w.part = x2.x, w.nP = uniform(x2.y), w.nt = uniform(x2.z), w.nb0 = uniform(x2.w);
        w.nb1 = uniform(x3.x), w.nb = uniform(x3.y), w.end = uniform(x3.z);
        return w.end == 0;
    };

    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kAtRegsIo));
        if (warp == 0 && lane == 0) {
            // ---------------------------------------------------------------- loads
            uint32_t it = 0, nq[2] = {0, 0};
            const uint32_t q_bytes = (uint32_t)(a.tpt * a.G * 128 * Sh::NKB);
            bool ok = !*abort_flag;
            const int heads = a.N * a.hkv_s, total = __ldcg(&a.ctl->n_wide) * heads;
            // The sorted list is taken from as CTAs become free, but for the first round; a few blocks before an item's
            // end, so that the next one's loads follow on.
            auto take = [&]() { return total > (int)gridDim.x ? (int)gridDim.x + atomicAdd(&a.ctl->next_wide, 1) : total; };
            auto publish = [&](int k, int& idx) {
                const int q = k % kAtQueue;
                if (idx >= total) idx = -1;
                AtWork w = {};
                w.end = 1;
                if (idx >= 0) {
                    const int e = idx / heads;
                    at_decode(a, e, idx - e * heads, w);
                }
                if (!(ok = at_wait(&item_empty[q], ((k / kAtQueue) & 1) ^ 1, abort_flag, a.status))) return;
                const int4* x = reinterpret_cast<const int4*>(&w);
                int4* y = reinterpret_cast<int4*>(&queue[q]);
#pragma unroll
                for (int i = 0; i < 4; ++i) y[i] = x[i];
                mbar_arrive(&item_full[q]);
            };
            int idx = blockIdx.x;
            if (ok) publish(0, idx);
            for (int k = 0; ok && idx >= 0; ++k) {
                const AtWork w = queue[k % kAtQueue];
                const int grp = w.b * a.hkv_s + w.kvh;
                auto load = [&](int j, bool v) {
                    bool own;
                    const int key0 = at_block(w, j, own);
                    const CUtensorMap* m = own ? (v ? &a.tv[w.r] : &a.tk[w.r]) : (v ? &a.pv[w.r] : &a.pk[w.r]);
                    const int s = it % R;
                    if (!(ok = at_wait(&kv_empty[s], ((it / R) & 1) ^ 1, abort_flag, a.status))) return;
                    mbar_arrive_expect_tx(&kv_full[s], Sh::KB);
#pragma unroll
                    for (int kb = 0; kb < Sh::NKB; ++kb)
                        tma_load_3d_keep(ring + s * Sh::KB + kb * (kAtK * 128), m, kb * 64, key0, own ? grp : w.kvh, &kv_full[s]);
                    ++it;
                };
                int in = 0;
                if (w.nb == 0) {
                    in = take();
                    publish(k + 1, in);
                }
                for (int j = 0; j < w.nb && ok; ++j) {
                    load(j, false);
                    if (j == max(0, w.nb - 4)) in = take();
                    if (j == 0) {
                        for (int t = 0; t < w.nt && ok; ++t) {
                            if ((t ? w.nb1 : w.nb0) == 0) continue;
                            if (!(ok = at_wait(&q_empty[t], (nq[t] & 1) ^ 1, abort_flag, a.status))) break;
                            mbar_arrive_expect_tx(&q_full[t], q_bytes);
#pragma unroll
                            for (int kb = 0; kb < Sh::NKB; ++kb)
                                tma_load_3d_keep(sq + t * Sh::QB + kb * (kAtM * 128), &a.tq, kb * 64, w.kvh * a.G,
                                                 w.r * a.T + w.t0 + t * a.tpt, &q_full[t]);
                            ++nq[t];
                        }
                    }
                    if (ok) load(j, true);
                    if (ok && j == max(0, w.nb - 2)) publish(k + 1, in);
                }
                idx = in;
            }
            volatile int no_abort = 0;      // no copy may still be landing when the CTA exits
            for (int t = 0; t < 2; ++t)
                if (nq[t]) mbar_wait(&q_full[t], (nq[t] - 1) & 1, &no_abort, nullptr);
            for (uint32_t k = it > (uint32_t)R ? it - R : 0; k < it; ++k)
                mbar_wait(&kv_full[k % R], (k / R) & 1, &no_abort, nullptr);
        } else if (warp == 1 || warp == 2) {
            // ---------------------------------------------------------------- products
            // A warp for each tile. The products queue only a few deep, so what a warp does between them is lost to the
            // tensor cores unless the other's are under way. They take turns, a block's products each: mixed with the
            // other's, a tile's would take twice as long, and both softmaxes would then wait and run together. The whole warp
            // runs the loop on warp-uniform values and one elected lane issues; the common block has a short path of its own.
            const int t = warp - 1;
            const uint32_t id_s = idesc_bf16(kAtM, kAtK), id_o = idesc_bf16_bmn(kAtM, D);
            const uint64_t dq = smem_desc_sw128(smem_u32(sq) + t * Sh::QB), dk0 = smem_desc_sw128(smem_u32(ring));
            const uint64_t dv0 = smem_desc_mn_sw128(smem_u32(ring), kAtK * 128, 1024);
            const uint32_t full0 = smem_u32(kv_full), empty0 = smem_u32(kv_empty), sf = smem_u32(&s_full[t]),
                           ph = smem_u32(&p_half[t]), pf = smem_u32(&p_full[t]);
            const uint32_t ts = tmem + kAtK * t, to = tmem + 2 * kAtK + D * t;
            uint32_t slot = 0, sph = 0;     // the ring's next slot and its phase
            uint32_t pp = 0, ip = 0, tp = 0, clean = 0;     // phases: blocks and items of the tile, turns, each slot's v_clean
            bool ok = true;
            auto wait_at = [&](uint32_t bar, uint32_t parity) {
                return (bool)__all_sync(0xffffffffu, mbar_try_at(bar, parity) || mbar_wait_slow(bar, parity, abort_flag, a.status));
            };
            const uint32_t mine = smem_u32(&turn[t]), other = smem_u32(&turn[1 - t]);
            auto take = [&]() { return wait_at(mine, (tp++ & 1) ^ (t == 0)); };
            auto pass = [&]() {
                if (lane == 0) asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(other) : "memory");
                __syncwarp();
            };
            auto release = [&]() {                          // once the products so far are done
                tc_commit_w(empty0 + 8 * slot);
                if (++slot == R) slot = 0, sph ^= 1;
            };
            auto issue_s = [&](bool last) {                 // S = Q K^T
                const uint64_t dk = at_desc_add(dk0, slot * Sh::KB);
#pragma unroll
                for (int kb = 0; kb < Sh::NKB; ++kb)
                    tc_mma4_w(ts, at_desc_add(dq, kb * (kAtM * 128)), at_desc_add(dk, kb * (kAtK * 128)), 2, 2, id_s, kb != 0);
                tc_commit_w(sf);
                if (last) tc_commit_w(smem_u32(&q_empty[t]));
            };
            auto issue_o = [&](bool first, int half) {      // O += P V, 64 of the 128 keys
                tc_mma4_ts_w(to, ts + 32 * half, at_desc_add(dv0, slot * Sh::KB + 8192 * half), 8, 128, id_o, !first);
            };
            AtWork w;
            for (int k = 0; ok && item(k, w); ++k) {
                if (!w.nb) continue;
                const int n = t ? w.nb1 : w.nb0, kend = at_kend(a, w);
                // blocks 1 .. plain - 1 are whole, seen by every row and followed by one of the tile; the prefix's last one
                // may be cut short
                const int own0 = w.nP - w.blk0;             // the item's first own block
                const int plain = min(n - 1, own0 + max(0, (w.qpos + 1) / kAtK));
                const int cut = a.prefix_len % kAtK ? own0 - 1 : -1;
                if (!(ok = wait_at(full0 + 8 * slot, sph))) break;
                if (n && !(ok = wait_at(smem_u32(&q_full[t]), ip & 1))) break;
                if (!(ok = take())) break;
                if (n) {
                    tc_fence_after();
                    issue_s(n == 1);
                }
                pass();
                release();
                for (int j = 0; j < w.nb; ++j) {
                    if (j >= 1 && j < plain && j != cut) {
                        const int stop = cut > j && cut < plain ? cut : plain;
                        while (true) {
                            const uint32_t sk = slot + 1 == R ? 0 : slot + 1;
                            if (!(ok = wait_at(full0 + 8 * slot, sph) && wait_at(full0 + 8 * sk, sk ? sph : sph ^ 1) &&
                                       wait_at(ph, pp & 1) && take())) break;
                            tc_fence_after();
                            issue_o(false, 0);
                            if (!(ok = wait_at(pf, pp & 1))) break;
                            tc_fence_after();
                            issue_o(false, 1);
                            ++pp;
                            release();
                            issue_s(j + 2 == n);
                            pass();
                            release();
                            if (++j == stop) break;
                        }
                        if (!ok) break;
                        --j;
                        continue;
                    }
                    bool own;
                    const int key0 = at_block(w, j, own);
                    if (!(ok = wait_at(full0 + 8 * slot, sph))) break;
                    if (own && at_ragged(w, key0)) {
                        if (!(ok = wait_at(smem_u32(&v_clean[slot]), clean >> slot & 1))) break;
                        clean ^= 1u << slot;
                    }
                    if (j < n) {
                        if (!(ok = wait_at(ph, pp & 1) && wait_at(pf, pp & 1))) break;
                        ++pp;
                        if (j == 0 && !(ok = wait_at(smem_u32(&o_empty[t]), (ip & 1) ^ 1))) break;
                    }
                    if (!(ok = take())) break;
                    if (j < n) {
                        tc_fence_after();
                        const int steps = (min(kAtK, (own ? kend : a.prefix_len) - key0) + 15) >> 4;
                        if (steps == kAtK / 16) {
                            issue_o(j == 0, 0);
                            issue_o(false, 1);
                        } else {
#pragma unroll 1
                            for (int kk = 0; kk < steps; ++kk)
                                tc_mma_ts_w(to, ts + 8 * kk, at_desc_add(dv0, slot * Sh::KB + kk * 16 * 128), id_o, (j | kk) != 0);
                        }
                        if (j + 1 == n) tc_commit_w(smem_u32(&o_full[t]));
                    }
                    release();
                    if (j + 1 < w.nb) {
                        if (!(ok = wait_at(full0 + 8 * slot, sph))) break;
                        if (j + 1 < n) {
                            tc_fence_after();
                            issue_s(j + 2 == n);
                        }
                        release();
                    }
                    pass();
                }
                if (n) ++ip;
            }
            tc_commit_w(smem_u32(done));
        } else if (warp == 3) {
            // ---------------------------------------------------------------- ragged V blocks
            // A consumer of every slot, so that it works as soon as a block has arrived and is never a round behind.
            uint32_t slot = 0, sph = 0;
            bool ok = true;
            auto next_slot = [&]() {
                __syncwarp();
                if (lane == 0) mbar_arrive(&kv_empty[slot]);
                if (++slot == R) slot = 0, sph ^= 1;
            };
            AtWork w;
            int k = 0;
            for (; ok && item(k, w, true); ++k) {
                const int kend = at_kend(a, w);
                int found = 0;
                for (int j = 0; j < w.nb; ++j) {
                    if (!(ok = __all_sync(0xffffffffu, at_wait(&kv_full[slot], sph, abort_flag, a.status)))) break;
                    next_slot();
                    if (!(ok = __all_sync(0xffffffffu, at_wait(&kv_full[slot], sph, abort_flag, a.status)))) break;
                    bool own;
                    const int key0 = at_block(w, j, own);
                    if (own && at_ragged(w, key0)) {
                        found |= v_block_finite<D>(ring + slot * Sh::KB, lane, min(kAtK, kend - key0));
                        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&v_clean[slot]);
                    }
                    next_slot();
                }
                if (!ok) break;
                found = __any_sync(0xffffffffu, found);
                if (lane == 0) {
                    s_poison[k % kAtQueue] = found;
                    mbar_arrive(&note[k % kAtQueue]);
                }
                item_done(k);
            }
        }
    } else if (warp < 12) {
        // -------------------------------------------------------------------- softmax
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kAtRegsSoftmax));
        const int t = (warp - 4) >> 2;                      // tile
        const int qd = warp & 3;                            // tensor-memory lane quarter
        const int m = 32 * qd + lane;                       // row of the tile
        const int tok = m / a.G + t * a.tpt;                // the row's token in the item
        const uint32_t lane_off = (uint32_t)(32 * qd) << 16;
        const uint32_t s_col = tmem + lane_off + kAtK * t, o_col = tmem + lane_off + 2 * kAtK + D * t;
        uint32_t sp = 0, ip = 0;                            // blocks, items of the tile so far
        bool ok = true;
        AtWork w;
        for (int k = 0; ok && item(k, w); ++k) {
            const int n = t ? w.nb1 : w.nb0;
            if (!n) continue;
            const int rows = min(a.tpt, w.ntok - t * a.tpt) * a.G;
            const bool idle = 32 * qd >= rows;              // a warp without rows only keeps the barriers' pace
            const int kend = at_kend(a, w);
            const int own_max = min((int64_t)kend - 1, (int64_t)w.qpos + tok);       // last own key the row sees
            const int warp_max = w.qpos + (32 * qd) / a.G + t * a.tpt;               // ... its warp's first row sees
            float m_use = -INFINITY, l_run = 0.f;
            for (int j = 0; j < n; ++j, ++sp) {
                ok = __all_sync(0xffffffffu, mbar_wait(&s_full[t], sp & 1, abort_flag, a.status));
                if (!ok) break;
                if (!idle) {
                    tc_fence_after();
                    bool own;
                    const int key0 = at_block(w, j, own);
                    // a block that every row of the warp sees whole needs no mask
                    const bool whole = own ? key0 + kAtK - 1 <= min(warp_max, kend - 1) : key0 + kAtK <= a.prefix_len;
                    const int hi = whole ? kAtK : (own ? own_max : a.prefix_len - 1) - key0;   // last key of the block the row sees
                    uint32_t v[4][32];
#pragma unroll
                    for (int c = 0; c < 4; ++c) tmem_ld32(s_col + 32 * c, v[c]);
                    tmem_wait_ld();
                    float* e = reinterpret_cast<float*>(&v[0][0]);
                    if (!whole) {
#pragma unroll
                        for (int i = 0; i < 128; ++i) e[i] = i <= hi ? e[i] : -INFINITY;
                    }
                    float mq[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};   // independent chains
#pragma unroll
                    for (int i = 0; i < 128; i += 2) mq[(i >> 1) & 3] = max3(mq[(i >> 1) & 3], e[i], e[i + 1]);
                    const float m_blk = fmaxf(fmaxf(mq[0], mq[1]), fmaxf(mq[2], mq[3])) * a.scale_log2;
                    const bool grow = m_blk > m_use + kAtRescale;
                    const float alpha = grow ? ex2_approx(m_use - m_blk) : 1.f;   // 0 when m_use is -inf
                    if (grow) m_use = m_blk;
                    // O holds the blocks before this one (their products precede this S in the
                    // order of issue); rescale it where the row's m moved
                    if (j > 0 && __any_sync(0xffffffffu, grow)) {
#pragma unroll 1
                        for (int c = 0; c < D / 16; ++c) {
                            uint32_t o[16];
                            tmem_ld16(o_col + 16 * c, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
                            tmem_st16(o_col + 16 * c, o);
                        }
                    }
                    const float m_sub = m_use == -INFINITY ? 0.f : m_use;         // nothing seen yet: every weight is 0
                    const uint64_t scale2 = f2_pack(a.scale_log2, a.scale_log2), neg2 = f2_pack(-m_sub, -m_sub);
                    uint64_t sum[4] = {0, 0, 0, 0};
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        uint32_t pk[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            float x, y;
                            f2_unpack(f2_fma(f2_pack(e[32 * c + 2 * i], e[32 * c + 2 * i + 1]), scale2, neg2), x, y);
                            x = ex2_approx(x);
                            y = ex2_approx(y);
                            sum[i & 3] = f2_add(sum[i & 3], f2_pack(x, y));
                            pk[i] = pack_bf16x2(x, y);
                        }
                        if (c == 2) {                       // the first 64 keys' products may begin
                            tmem_wait_st();
                            tc_fence_before();
                            __syncwarp();
                            if (lane == 0) mbar_arrive(&p_half[t]);
                        }
                        tmem_st16(s_col + 16 * c, pk);
                    }
                    float sx, sy;
                    f2_unpack(f2_add(f2_add(sum[0], sum[1]), f2_add(sum[2], sum[3])), sx, sy);
                    l_run = l_run * alpha + (sx + sy);
                    tmem_wait_st();
                    tc_fence_before();
                } else {
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&p_half[t]);
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_full[t]);
            }
            if (!ok) break;
            ok = __all_sync(0xffffffffu, mbar_wait(&st_empty[t], (ip & 1) ^ 1, abort_flag, a.status));
            if (!ok) break;
            stat[t * kAtM + m] = make_float2(m_use, l_run);
            ++ip;
            __syncwarp();
            if (lane == 0) mbar_arrive(&st_full[t]);
        }
    } else {
        // -------------------------------------------------------------------- results
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kAtRegsOut));
        const int qd = warp & 3, m = 32 * qd + lane;
        const int tok0 = m / a.G, g = m - tok0 * a.G;
        const uint32_t o_col = tmem + ((uint32_t)(32 * qd) << 16) + 2 * kAtK;
        uint32_t ip0 = 0, ip1 = 0;
        bool ok = true;
        for (int k = 0; ok; ++k) {
            AtWork w;
            if (!item(k, w, true)) break;
            const int ntok = w.ntok, qpos = w.qpos;
            const bool part = w.part >= 0;
            const int rows = ntok * a.G;
            // the item's first row of results, moved to the unit that the lane stores
            const int64_t prow = (int64_t)w.part + (int64_t)w.h * rows;
            char* base = part ? reinterpret_cast<char*>(a.part_o + prow * D)
                              : reinterpret_cast<char*>(a.out + (((int64_t)w.r * a.T + w.t0) * a.hq_s + w.kvh * a.G) * D);
            base += (lane & 3) * 16;
            const int row_bytes = part ? D * 4 : D * 2, tok_rows = part ? a.G : a.hq_s;
            int poison = 0;
#pragma unroll 1
            for (int t = 0; t < w.nt && ok; ++t) {
                const int n = t ? w.nb1 : w.nb0, tok = tok0 + t * a.tpt;
                const bool live = tok0 < a.tpt && tok < ntok;
                const int64_t pos = (int64_t)qpos + tok;
                float2 ml = make_float2(-INFINITY, 0.f);
                if (n) {
                    const uint32_t ph = (t ? ip1 : ip0) & 1;
                    // the item's notes are there by then: a product waits for them
                    ok = __all_sync(0xffffffffu, mbar_wait(&st_full[t], ph, abort_flag, a.status) &&
                                                     mbar_wait(&o_full[t], ph, abort_flag, a.status) &&
                                                     mbar_wait(&note[k % kAtQueue], (k / kAtQueue) & 1, abort_flag, a.status));
                    if (!ok) break;
                    if (t) ++ip1;
                    else ++ip0;
                    tc_fence_after();
                    ml = stat[t * kAtM + m];
                    poison |= s_poison[k % kAtQueue];
                }
                const bool zero = !n || (!part && (pos < 0 || pos >= a.max_kv));
                const float f = zero ? 0.f : part ? 1.f : 1.f / ml.y;
                if (part && live) a.part_ml[prow + tok * a.G + g] = ml;
                const unsigned store = __ballot_sync(0xffffffffu, live) >> (lane & 28);
                const int row = (tok * tok_rows + g) * row_bytes;
                int to[4];                                  // the four rows whose units the lane stores
#pragma unroll
                for (int i = 0; i < 4; ++i) to[i] = __shfl_sync(0xffffffffu, row, (lane & 28) | i);
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
                    uint32_t o[32];
                    if (n) tmem_ld32(col, o);
#pragma unroll 1
                    for (int c = 0; c < D / 32; ++c) {
                        uint4 u[4] = {};
                        if (n) {
                            tmem_wait_ld();
                            if (!zero) {
#pragma unroll
                                for (int i = 0; i < 4; ++i)
                                    u[i] = make_uint4(pack_bf16x2(__uint_as_float(o[8 * i]) * f, __uint_as_float(o[8 * i + 1]) * f),
                                                      pack_bf16x2(__uint_as_float(o[8 * i + 2]) * f, __uint_as_float(o[8 * i + 3]) * f),
                                                      pack_bf16x2(__uint_as_float(o[8 * i + 4]) * f, __uint_as_float(o[8 * i + 5]) * f),
                                                      pack_bf16x2(__uint_as_float(o[8 * i + 6]) * f, __uint_as_float(o[8 * i + 7]) * f));
                            }
                            if (c + 1 < D / 32) tmem_ld32(col + 32 * c + 32, o);
                            transpose4(u, lane);
                        }
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (store >> i & 1) *reinterpret_cast<uint4*>(base + to[i] + 64 * c) = u[i];
                    }
                }
                if (n) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(&o_empty[t]);
                        mbar_arrive(&st_empty[t]);
                    }
                }
            }
            if (ok && poison) {                             // what the rows do see of the values that are not finite
                __syncwarp();
                const AtWork* q = &queue[k % kAtQueue];
                for (int t = 0; t < q->nt; ++t) {
                    const int tok = tok0 + t * a.tpt;
                    const int64_t pos = (int64_t)q->qpos + tok;
                    if (tok0 >= a.tpt || tok >= q->ntok || pos >= a.max_kv) continue;
                    const int end = (int)min((int64_t)at_kend(a, *q) - 1, pos);
                    const int ragged = max(0, (q->qpos + 1) / kAtK) * kAtK, first = max(0, q->blk0 - q->nP) * kAtK;
                    const bf16* v = a.v[q->r] + ((int64_t)q->b * a.hkv_s + q->kvh) * a.max_kv * D;
                    float* po = a.part_o + ((int64_t)q->part + (int64_t)q->h * q->ntok * a.G + tok * a.G + g) * D;
                    bf16* out = a.out + (((int64_t)q->r * a.T + q->t0 + tok) * a.hq_s + q->kvh * a.G + g) * D;
#pragma unroll 1
                    for (int key = max(ragged, first); key <= end; ++key)
#pragma unroll 1
                        for (int i = 0; i < D; ++i) {
                            const float x = __bfloat162float(v[(int64_t)key * D + i]);
                            if (fabsf(x) < INFINITY) continue;
                            if (q->part >= 0) po[i] += x;
                            else out[i] = __float2bfloat16_rn(__bfloat162float(out[i]) + x);
                        }
                }
            }
            if (ok) item_done(k);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        volatile int no_abort = 0;                   // every MMA has retired before the columns are freed
        mbar_wait(done, 0, &no_abort, nullptr);
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, 512);
        tmem_relinquish();
    }
}

// ---------------------------------------------------------------------------
// Items of at most 32 query rows (single tokens, most of a decode step): bound
// by the bytes of K and V. With the queries as the rows of a tile, a product
// would be mostly padding and a row's softmax the work of one thread; so the
// keys are the rows: S^T = K Q^T (128 keys x 16 or 32 rows), and O^T = V^T P^T
// (d x rows) with V read as the M-major operand and P^T from shared memory. A
// thread has one key: its scores of every row are one column each. A CTA works
// at two items at a time, in two halves with a ring each that cover one
// another's waits (a kernel that allocates tensor memory gets one CTA per SM).
// Of each half's eight warps
//   warps 0-3   the softmax of a block, one key per thread: maxima over the
//               keys by redux and one exchange between the warps; P^T to shared
//               memory in bf16; the previous block's O^T (one element of d per
//               thread) from tensor memory to registers. m moves as in the wide
//               kernel. The V rows that some row does not see are made finite
//               by the thread of the key.
//   warp 4      takes the items from the list as the half becomes free, TMA
//   warp 5      products
//   warps 6, 7  nothing (registers are dealt out to groups of four warps)
// Decode of 256 sequences of 0 to 2047 keys behind 16384 shared ones, 32 heads:
// 1.15 GB in 198 to 203 us, 5.7 to 5.8 TB/s, the shared keys on the wide kernel
// beside it and the joining included. Taking the items out of tiles of 128 query
// rows took that call from 473 to 305 us, the two halves from 271 to 242.
// This kernel's own reading goes at the measured copy rate (6.8 TB/s in 171 us).
// ---------------------------------------------------------------------------

constexpr int kAnThreads = 512, kAnHalf = 256;   // of a half's two warpgroups the second gives registers to the first
constexpr int kAnRegsIo = 80, kAnRegsSoftmax = 176;
static_assert(kAnRegsIo + kAnRegsSoftmax <= 2 * 128, "the launch's registers");
constexpr int kAnQueue = 4;               // items taken ahead
// Keys per TMA box: a sequence's last block brings no more of them than it must. Decode of 256 sequences of 0 to 2047 keys
// of their own 205 us with boxes of 128, 201 with 32, 202 with 64, 206 with 16; of 64 of 1000 each, whose last block is
// nearly full, 55.6, 56.9, 56.3 and 58.0.
constexpr int kAnBox = 32;

template <int D>
struct AnShape {
    static constexpr int NKB = D / 64;
    static constexpr int KB = kAtK * D * 2;
    static constexpr int RING = D == 128 ? 3 : 6;
    static constexpr int HEAD = 1024;                   // barriers, the queue, the warps' maxima
    static constexpr int QB = kAtNarrow * D * 2;
    static constexpr int PB = kAtNarrow * kAtK * 2;
    // a block of 64-element V rows is read as if it had 128: the other half is whatever follows, up to KB bytes on
    static constexpr int PAD = D == 64 ? KB - QB - PB : 0;
    static constexpr int SMEM = RING * KB + QB + PB + PAD + HEAD;
};
static_assert(2 * AnShape<128>::SMEM + 1024 <= 227 * 1024 && 2 * AnShape<64>::SMEM + 1024 <= 227 * 1024, "two halves");
static_assert(AnShape<128>::SMEM % 1024 == 0 && AnShape<64>::SMEM % 1024 == 0, "alignment of the second");

__device__ __forceinline__ float redux_max(float v) {
    float r;
    asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
}

template <int D>
struct AnCtx {
    const AtArgs* a;
    int tid;                              // thread of the half's softmax
    unsigned char *ring, *p;
    uint64_t *s_full, *p_full, *o_full, *x_full, *x_empty, *v_ragged;
    float* wmax;                          // [4][kAtNarrow]
    volatile int *abort_flag, *s_poison;
    uint32_t tmem, base, blocks, ragged, exchanges;   // base: ring index of the item's first block
    int np;
};

// An item's softmax and results for NR = 4, 8, 16 or 32 rows (of the 16 or 32 of the products); false: a wait gave up.
template <int D, int NR>
__device__ __forceinline__ bool an_item(AnCtx<D>& c, const AtWork& w) {
    using Sh = AnShape<D>;
    const AtArgs& a = *c.a;
    const int tid = c.tid, warp = tid >> 5, lane = tid & 31;
    const int rows = w.ntok * a.G, kend = at_kend(a, w);
    const uint32_t lane_off = (uint32_t)(32 * warp) << 16;
    float o[NR], l[NR];
#pragma unroll
    for (int n = 0; n < NR; ++n) o[n] = l[n] = 0.f;
    float m_lane = -INFINITY, alpha_prev = 1.f;          // lane n: row n's m, and what it changed by in the last block
    bool moved_prev = false;
    int first_ragged = INT_MAX, poison = 0;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
        return (bool)__all_sync(0xffffffffu, mbar_wait(bar, parity, c.abort_flag, a.status));
    };
    // every warp's value of row n to lane n of all
    auto exchange = [&](float mine, float (&x)[4]) {
        if (!wait(c.x_empty, (c.exchanges & 1) ^ 1)) return false;
        if (lane < NR) c.wmax[warp * kAtNarrow + lane] = mine;
        __syncwarp();
        if (lane == 0) mbar_arrive(c.x_full);
        if (!wait(c.x_full, c.exchanges & 1)) return false;
        ++c.exchanges;
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = *const_cast<volatile float*>(&c.wmax[i * kAtNarrow + (lane & (NR - 1))]);
        __syncwarp();
        if (lane == 0) mbar_arrive(c.x_empty);
        return true;
    };
    auto take_o = [&]() {                                // the last block's product onto the running sums
        uint32_t x[NR];
        if constexpr (NR == 32) tmem_ld32(c.tmem + 64 + lane_off, x);
        else if constexpr (NR == 16) tmem_ld16(c.tmem + 64 + lane_off, x);
        else if constexpr (NR == 8) tmem_ld8(c.tmem + 64 + lane_off, x);
        else tmem_ld4(c.tmem + 64 + lane_off, x);
        tmem_wait_ld();
        if (moved_prev) {
#pragma unroll
            for (int n = 0; n < NR; ++n)
                o[n] = fmaf(o[n], __shfl_sync(0xffffffffu, alpha_prev, n), __uint_as_float(x[n]));
        } else {
#pragma unroll
            for (int n = 0; n < NR; ++n) o[n] += __uint_as_float(x[n]);
        }
    };
    for (int j = 0; j < w.nb; ++j, ++c.blocks) {
        if (!wait(&c.s_full[c.blocks & 1], (c.blocks >> 1) & 1)) return false;
        tc_fence_after();
        uint32_t v[NR];
        if constexpr (NR == 32) tmem_ld32(c.tmem + 32 * (c.blocks & 1) + lane_off, v);
        else if constexpr (NR == 16) tmem_ld16(c.tmem + 32 * (c.blocks & 1) + lane_off, v);
        else if constexpr (NR == 8) tmem_ld8(c.tmem + 32 * (c.blocks & 1) + lane_off, v);
        else tmem_ld4(c.tmem + 32 * (c.blocks & 1) + lane_off, v);
        tmem_wait_ld();
        bool own;
        const int key0 = at_block(w, j, own), key = key0 + tid;
        // the first row that sees the thread's key
        int first = 0;
        if (own) first = key >= kend ? NR : (int)max((int64_t)0, min((int64_t)NR, ((int64_t)key - w.qpos) * a.G));
        else if (key >= a.prefix_len) first = NR;
        float mine = -INFINITY;
#pragma unroll
        for (int n = 0; n < NR; ++n) {
            const float s = n >= first ? __uint_as_float(v[n]) : -INFINITY;
            v[n] = __float_as_uint(s);
            const float r = redux_max(s);
            if (lane == n) mine = r;
        }
        float x[4];
        if (!exchange(mine, x)) return false;
        const float m_blk = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])) * a.scale_log2;
        const bool grow = m_blk > m_lane + kAtRescale;
        const float alpha = grow ? ex2_approx(m_lane - m_blk) : 1.f;
        if (grow) m_lane = m_blk;
        const bool moved = __any_sync(0xffffffffu, grow);
        const float m_sub = m_lane == -INFINITY ? 0.f : m_lane;
        if (moved)
#pragma unroll
            for (int n = 0; n < NR; ++n) l[n] *= __shfl_sync(0xffffffffu, alpha, n);
#pragma unroll
        for (int n = 0; n < NR; ++n) {
            const float e = ex2_approx(fmaf(__uint_as_float(v[n]), a.scale_log2, -__shfl_sync(0xffffffffu, m_sub, n)));
            l[n] += e;
            v[n] = __float_as_uint(e);
        }
        if (j > 0) {                                     // also: the products no longer read P^T
            if (!wait(c.o_full, (c.blocks - 1) & 1)) return false;
            tc_fence_after();
            take_o();
        }
        alpha_prev = alpha;
        moved_prev = moved;
        // P^T: 64 keys per 128-byte row of one query row, rows in atoms of 8, 16-byte units swizzled
        unsigned char* pr = c.p + (tid >> 6) * (kAtNarrow * 128) + (tid & 7) * 2;
        const int unit = (tid & 63) >> 3;
#pragma unroll
        for (int n = 0; n < NR; ++n)
            *reinterpret_cast<bf16*>(pr + n * 128 + ((unit ^ (n & 7)) << 4)) = __float2bfloat16_rn(__uint_as_float(v[n]));
        if (own && at_ragged(w, key0)) {
            if (!wait(c.v_ragged, c.ragged & 1)) return false;
            ++c.ragged;
            first_ragged = min(first_ragged, key0);
            // K and V of a block: K_0 K_1 V_0 K_2 V_1 ... V_last
            const uint32_t iv = c.base + (j + 1 < w.nb ? 2 * j + 2 : 2 * j + 1);
            const int hit = v_row_finite<D>(c.ring + (iv % Sh::RING) * Sh::KB, tid, key >= kend);
            if (__any_sync(0xffffffffu, hit) && lane == 0) c.s_poison[c.np & 1] = c.np + 1;
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(c.p_full);
    }
    c.base += 2 * w.nb;
    float l_lane = 0.f;
    if (w.nb) {
        if (!wait(c.o_full, (c.blocks - 1) & 1)) return false;
        tc_fence_after();
        take_o();
        tc_fence_before();
        // sums over the keys: each step halves the rows a lane holds; lane n ends with row n's
#pragma unroll
        for (int off = NR / 2; off; off >>= 1) {
            const bool up = lane & off;
#pragma unroll
            for (int n = 0; n < off; ++n) {
                const float keep = up ? l[n + off] : l[n], give = up ? l[n] : l[n + off];
                l[n] = keep + __shfl_xor_sync(0xffffffffu, give, off);
            }
        }
#pragma unroll
        for (int off = NR; off < 32; off *= 2) l[0] += __shfl_xor_sync(0xffffffffu, l[0], off);
        float x[4];
        if (!exchange(l[0], x)) return false;
        l_lane = (x[0] + x[1]) + (x[2] + x[3]);
        if (first_ragged != INT_MAX) {
            poison = c.s_poison[c.np & 1] == c.np + 1;
            ++c.np;
        }
        if (poison && tid < D) {                         // what the rows do see of the values that are not finite
            const bf16* v = a.v[w.r] + ((int64_t)w.b * a.hkv_s + w.kvh) * a.max_kv * D + tid;
            for (int key = first_ragged; key < kend; ++key) {
                const float x = __bfloat162float(v[(int64_t)key * D]);
                if (fabsf(x) < INFINITY) continue;
                const int64_t first = ((int64_t)key - w.qpos) * a.G;
#pragma unroll
                for (int n = 0; n < NR; ++n)
                    if (n >= first) o[n] += x;
            }
        }
    }
    if (w.part >= 0) {
        const int64_t row0 = (int64_t)w.part + (int64_t)w.h * rows;
        if (warp == 0 && lane < rows) a.part_ml[row0 + lane] = make_float2(m_lane, l_lane);
        if (tid < D) {
            float* dst = a.part_o + row0 * D + tid;
#pragma unroll
            for (int n = 0; n < NR; ++n)
                if (n < rows) dst[n * D] = o[n];
        }
        return true;
    }
    const int64_t pos = (int64_t)w.qpos + lane / a.G;    // lane n: row n's
    const float inv = pos >= 0 && pos < a.max_kv ? 1.f / l_lane : 0.f;
    const unsigned zero = __ballot_sync(0xffffffffu, pos < 0 || pos >= a.max_kv);
    bf16* dst = a.out + (((int64_t)w.r * a.T + w.t0) * a.hq_s + w.kvh * a.G) * D + tid;
    int g = 0;
#pragma unroll
    for (int n = 0; n < NR; ++n) {
        const float f = __shfl_sync(0xffffffffu, inv, n);
        if (n < rows && tid < D) dst[(int64_t)g * D] = __float2bfloat16_rn((zero >> n & 1) ? 0.f : o[n] * f);
        if (++g == a.G) {
            g = 0;
            dst += (int64_t)a.hq_s * D;
        }
    }
    return true;
}

// The plan of a call of so few rows that all items are narrow and its fewer than
// 32 sequences have one tile each: a lane per sequence, the lane behind them for
// the tile of a shared prefix. Every CTA makes it for itself, without the
// plan kernel and the way from it to here: 4 tokens behind 777 shared rows take
// 13 us from the first kernel's start to the last one's end, and took 22. The
// items are dealt out in turn.
struct AnFew {
    int before[32];                       // items in front of the lane's
    int t0[32], ntok[32], qpos[32], nb[32], len[32], row1[32];
    int total, reserved[31];
};
static_assert(sizeof(AnFew) == 1024, "behind the two halves");

// One warp. record: this CTA's also writes what the joining kernel reads, and the status.
__device__ __noinline__ void an_few_plan(const AtArgs& a, AnFew* f, int lane, bool record) {
    constexpr unsigned kAll = 0xffffffffu;
    const int heads = a.N * a.hkv_s;
    int c = 0, c1 = 0, n = 0, q = 0;
    bool bad = false, out = false;
    if (lane < a.B) {
        c = a.cu[lane];
        c1 = a.cu[lane + 1];
        q = a.pos[lane];
        bad = c1 < c || c < 0 || c1 > a.T || (lane == 0 && c != 0);
        n = c1 - c;
        out = n > 0 && (q < 0 || (int64_t)q + n > a.max_kv);
    }
    bad = __any_sync(kAll, bad);
    out = __any_sync(kAll, out);
    const int n_tok = __shfl_sync(kAll, c1, a.B - 1);
    const bool prefix = lane == a.B && a.prefix_len;
    if (prefix) n = n_tok;
    if (bad) n = 0;
    const int nb = !n ? 0 : prefix ? (a.prefix_len + kAtK - 1) / kAtK : own_blocks((int64_t)q + n, a.max_kv);
    int parts, len;
    part_split(nb, narrow_share((unsigned)__reduce_add_sync(kAll, nb), heads), false, parts, len);
    if (!n) parts = 0;
    const int items = warp_scan(parts, lane), more = max(parts - 1, 0) * heads * n * a.G;
    const int row1 = 2 * a.T * heads * a.G + warp_scan(more, lane) - more;
    f->before[lane] = items - parts;
    f->t0[lane] = c;
    f->ntok[lane] = n;
    f->qpos[lane] = q;
    f->nb[lane] = nb;
    f->len[lane] = len;
    f->row1[lane] = row1;
    if (lane == 31) f->total = items;
    if (!record) return;
    const int chunks = n && !prefix && (parts > 1 || a.prefix_len) ? (n * a.G + 7) / 8 : 0;
    const int upto = warp_scan(chunks, lane), sum = __shfl_sync(kAll, upto, 31);
    for (int j = 0; j < chunks; ++j) a.chunks[upto - chunks + j] = AttnChunk{c, n, q, row1, parts, j, 0, 0};
    if (prefix) a.prefix_groups[0] = make_int2(row1, parts);
    if (lane == 0) {
        AttnCtl x = {};
        x.n_tokens = bad ? 0 : n_tok;
        x.n_chunks = sum;
        *a.ctl = x;
        if (bad) set_status(a.status, TP_ERR_SHAPE);
        else if (out) set_status(a.status, TP_ERR_CAPACITY);
    }
}

// item e of the few
__device__ __forceinline__ void an_few_item(const AtArgs& a, const AnFew* f, int e, int4& x, int4& y) {
    int l = 0;
#pragma unroll 1
    for (int o = 16; o; o >>= 1)
        if (f->before[l + o] <= e) l += o;
    const int j = e - f->before[l], end = l < 31 ? f->before[l + 1] : f->total, parts = end - f->before[l], len = f->len[l];
    const bool prefix = l == a.B;
    const int rows = a.N * a.hkv_s * a.G;
    int row = -1;
    if (parts > 1 || a.prefix_len) row = j ? f->row1[l] + (j - 1) * rows * f->ntok[l] : rows * ((prefix ? a.T : 0) + f->t0[l]);
    x = make_int4(f->t0[l], f->ntok[l], l, f->qpos[l]);
    y = make_int4(j * len, min(f->nb[l], (j + 1) * len), prefix ? AT_PREFIX : AT_OWN, row);
}

template <int D>
__global__ void __launch_bounds__(kAnThreads, 1) attn_narrow_kernel(const __grid_constant__ AtArgs a) {
    using Sh = AnShape<D>;
    constexpr int R = Sh::RING;
    extern __shared__ __align__(1024) unsigned char smem[];
    const int half = uniform(threadIdx.x / kAnHalf);
    unsigned char* ring = smem + half * Sh::SMEM;
    unsigned char* sq = ring + R * Sh::KB;
    unsigned char* sp = sq + Sh::QB;
    unsigned char* head = sp + Sh::PB + Sh::PAD;
    uint64_t* bars = reinterpret_cast<uint64_t*>(head);
    uint64_t* kv_full = bars;             // [R]
    uint64_t* kv_empty = kv_full + R;     // [R]
    uint64_t* q_full = kv_empty + R;
    uint64_t* q_empty = q_full + 1;
    uint64_t* s_full = q_empty + 1;       // [2]
    uint64_t* p_full = s_full + 2;
    uint64_t* o_full = p_full + 1;
    uint64_t* x_full = o_full + 1;        // the warps' maxima or sums are there
    uint64_t* x_empty = x_full + 1;       // ... and read
    uint64_t* v_ragged = x_empty + 1;
    uint64_t* item_full = v_ragged + 1;   // [kAnQueue]
    uint64_t* item_empty = item_full + kAnQueue;
    uint64_t* done = item_empty + kAnQueue;
    int* queue = reinterpret_cast<int*>(done + 1);                   // [kAnQueue]
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(queue + kAnQueue);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    volatile int* s_poison = reinterpret_cast<volatile int*>(tmem_slot + 2);   // [2]
    float* wmax = reinterpret_cast<float*>(head + Sh::HEAD - 4 * kAtNarrow * 4);
    int4* entry = reinterpret_cast<int4*>(wmax) - 2 * kAnQueue;      // [kAnQueue][2]: the queue's items as they are listed
    static_assert((2 * R + 9 + 2 * kAnQueue + 1) * 8 + (kAnQueue + 4) * 4 <= Sh::HEAD - 4 * kAtNarrow * 4 - 32 * kAnQueue,
                  "the head's words");

    const int tid = threadIdx.x % kAnHalf, warp = uniform(tid >> 5), lane = tid & 31;
    // Behind the wide kernel the lists are there: it lets this one start only after its own wait. This kernel waits for
    // the wide one at its end, so that what follows it follows both. Often there is nothing left for it.
    int n_wide = 0, n_items = 0;
    if (a.after_wide) {
        n_wide = __ldcg(&a.ctl->n_wide);
        n_items = __ldcg(&a.ctl->n_items);
    }
    if (tid == 0) {
        for (int i = 0; i < R; ++i) {
            mbar_init(&kv_full[i], 1);
            mbar_init(&kv_empty[i], 1);
        }
        mbar_init(q_full, 1);
        mbar_init(q_empty, 1);
        mbar_init(&s_full[0], 1);
        mbar_init(&s_full[1], 1);
        mbar_init(p_full, 4);
        mbar_init(o_full, 1);
        mbar_init(x_full, 4);
        mbar_init(x_empty, 4);
        mbar_init(v_ragged, 1);
        for (int i = 0; i < kAnQueue; ++i) {
            mbar_init(&item_full[i], 1);
            mbar_init(&item_empty[i], 5);
        }
        mbar_init(done, 1);
        *abort_flag = (smem_u32(ring) & 1023u) ? 1 : 0;
        s_poison[0] = s_poison[1] = 0;
        if (*abort_flag) set_status(a.status, TP_ERR_ALIGN);
        fence_mbar_init();
    }
    if (a.after_wide && n_items == n_wide) {
        pdl_trigger();
        pdl_wait();
        return;
    }
    if (warp == 5 && half == 0) tmem_alloc(smem_u32(tmem_slot), 256);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = uniform(*reinterpret_cast<uint32_t*>(reinterpret_cast<unsigned char*>(tmem_slot) - half * Sh::SMEM)) + 128 * half;
    if (!a.after_wide) pdl_wait();
    pdl_trigger();
    const int heads = a.N * a.hkv_s;
    AnFew* few = reinterpret_cast<AnFew*>(smem + 2 * Sh::SMEM);
    int total;
    if (a.few) {
        if (threadIdx.x < 32) an_few_plan(a, few, lane, blockIdx.x == gridDim.x - 1);
        __syncthreads();
        total = few->total * heads;
    } else {
        if (!a.after_wide) n_items = __ldcg(&a.ctl->n_items);         // none is wide
        total = (n_items - n_wide) * heads;
    }
    if (*abort_flag) total = 0;
    // the i-th item of this CTA, -1 when there are no more
    auto item = [&](int i, AtWork& w, bool& more) {
        const int s = i % kAnQueue;
        bool ok = __all_sync(0xffffffffu, mbar_wait(&item_full[s], (i / kAnQueue) & 1, abort_flag, a.status));
        if (!ok) return false;
        const int idx = *reinterpret_cast<volatile int*>(&queue[s]);
        const int4 x = entry[2 * s], y = entry[2 * s + 1];
        __syncwarp();
        if (lane == 0) mbar_arrive(&item_empty[s]);
        more = idx >= 0;
        if (more) at_fill(a, x, y, idx % heads, w);
        return true;
    };

    if (warp >= 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kAnRegsIo));
        if (warp == 4 && lane == 0) {
            uint32_t it = 0, nq = 0;        // loads, Q tiles
            const uint32_t q_bytes = (uint32_t)(kAtNarrow / a.G * a.G * 128 * Sh::NKB);
            bool ok = !*abort_flag;
            // As the wide kernel's, the first one too: behind that kernel the CTAs start as its CTAs end.
            int turn = blockIdx.x + half * gridDim.x;
            auto take = [&]() {
                if (!a.few) return total ? atomicAdd(&a.ctl->next, 1) : 0;
                const int idx = turn;
                if (turn < total) turn += 2 * gridDim.x;
                return idx;
            };
            auto publish = [&](int i, int& idx, AtWork& w) {
                const int s = i % kAnQueue;
                if (idx >= total) idx = -1;
                const int e = idx / heads;
                int4 x = {}, y = {};
                if (idx >= 0) {
                    if (a.few) an_few_item(a, few, e, x, y);
                    else at_load(a, n_wide + e, x, y);
                }
                if (!(ok = mbar_wait(&item_empty[s], ((i / kAnQueue) & 1) ^ 1, abort_flag, a.status))) return;
                *reinterpret_cast<volatile int*>(&queue[s]) = idx;
                entry[2 * s] = x;
                entry[2 * s + 1] = y;
                mbar_arrive(&item_full[s]);
                if (idx >= 0) at_fill(a, x, y, idx - e * heads, w);
            };
            AtWork w, wn;
            int idx = -1, in = 0;
            if (ok) {
                idx = take();
                publish(0, idx, w);
            }
            for (int i = 0; ok && idx >= 0; ++i) {
                const int grp = w.b * a.hkv_s + w.kvh, kend = at_kend(a, w);
                auto load = [&](int j, bool v) {
                    bool own;
                    const int key0 = at_block(w, j, own);
                    const CUtensorMap* m = own ? (v ? &a.tv[w.r] : &a.tk[w.r]) : (v ? &a.pv[w.r] : &a.pk[w.r]);
                    const int sl = it % R;
                    if (!(ok = mbar_wait(&kv_empty[sl], ((it / R) & 1) ^ 1, abort_flag, a.status))) return;
                    // the rows behind the last box are not read: their scores are masked, and the products with V end with
                    // the last 16 keys in use
                    const int boxes = (min(kAtK, (own ? kend : a.prefix_len) - key0) + kAnBox - 1) / kAnBox;
                    mbar_arrive_expect_tx(&kv_full[sl], boxes * kAnBox * D * 2);
#pragma unroll 1
                    for (int i = 0; i < boxes; ++i)
#pragma unroll
                        for (int kb = 0; kb < Sh::NKB; ++kb)
                            tma_load_3d_keep(ring + sl * Sh::KB + kb * (kAtK * 128) + i * (kAnBox * 128), m, kb * 64,
                                             key0 + i * kAnBox, own ? grp : w.kvh, &kv_full[sl]);
                    ++it;
                };
                if (w.nb) {
                    load(0, false);
                    if (ok && (ok = mbar_wait(q_empty, (nq & 1) ^ 1, abort_flag, a.status))) {
                        mbar_arrive_expect_tx(q_full, q_bytes);
#pragma unroll
                        for (int kb = 0; kb < Sh::NKB; ++kb)
                            tma_load_3d_keep(sq + kb * (kAtNarrow * 128), &a.tqn, kb * 64, w.kvh * a.G, w.r * a.T + w.t0, q_full);
                        ++nq;
                    }
                }
                if (!ok) break;
                if (w.nb == 0) {
                    in = take();
                    publish(i + 1, in, wn);
                }
                for (int j = 0; j < w.nb && ok; ++j) {
                    if (j == max(0, w.nb - 3)) in = take();
                    if (j + 1 < w.nb) load(j + 1, false);
                    if (ok && j == max(0, w.nb - 2)) publish(i + 1, in, wn);
                    if (ok) load(j, true);
                }
                w = wn;
                idx = in;
            }
            volatile int no_abort = 0;      // no copy may still be landing when the CTA exits
            if (nq) mbar_wait(q_full, (nq - 1) & 1, &no_abort, nullptr);
            for (uint32_t k = it > (uint32_t)R ? it - R : 0; k < it; ++k)
                mbar_wait(&kv_full[k % R], (k / R) & 1, &no_abort, nullptr);
        } else if (warp == 5) {
            const uint64_t dq = smem_desc_sw128(smem_u32(sq)), dk0 = smem_desc_sw128(smem_u32(ring)), dp = smem_desc_sw128(smem_u32(sp));
            const uint64_t dv0 = smem_desc_mn_sw128(smem_u32(ring), kAtK * 128, 1024);
            uint32_t it = 0, blocks = 0, nq = 0;
            bool ok = !*abort_flag, more = true;
            auto wait_all = [&](uint64_t* bar, uint32_t parity) {
                return (bool)__all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, a.status));
            };
            AtWork w;
            for (int i = 0; ok; ++i) {
                if (!(ok = item(i, w, more)) || !more) break;
                if (!w.nb) continue;
                const int nr = w.ntok * a.G <= 16 ? 16 : 32;
                const uint32_t id_s = idesc_bf16(kAtK, nr), id_o = idesc_bf16_amn(128, nr);
                auto issue_s = [&](int j) {                  // S^T of block j into the buffer of its turn
                    const uint32_t s = it % R;
                    if (!(ok = wait_all(&kv_full[s], (it / R) & 1))) return;
                    ++it;
                    tc_fence_after();
                    const uint64_t dk = at_desc_add(dk0, s * Sh::KB);
    #pragma unroll
                    for (int kb = 0; kb < Sh::NKB; ++kb)
    #pragma unroll
                        for (int k = 0; k < 4; ++k)
                            tc_mma_w(tmem + 32 * ((blocks + j) & 1), at_desc_add(dk, kb * (kAtK * 128) + k * 32),
                                     at_desc_add(dq, kb * (kAtNarrow * 128) + k * 32), id_s, (kb | k) != 0);
                    tc_commit_w(smem_u32(&s_full[(blocks + j) & 1]));
                    tc_commit_w(smem_u32(&kv_empty[s]));
                    if (j + 1 == w.nb) tc_commit_w(smem_u32(q_empty));
                };
                if (!(ok = wait_all(q_full, nq & 1))) break;
                ++nq;
                issue_s(0);
                for (int j = 0; j < w.nb && ok; ++j) {
                    if (j + 1 < w.nb) issue_s(j + 1);
                    if (!ok) break;
                    const uint32_t s = it % R;
                    if (!(ok = wait_all(&kv_full[s], (it / R) & 1))) break;
                    ++it;
                    bool own;
                    const int key0 = at_block(w, j, own);
                    if (own && at_ragged(w, key0) && lane == 0) mbar_arrive(v_ragged);
                    __syncwarp();
                    if (!(ok = wait_all(p_full, (blocks + j) & 1))) break;
                    tc_fence_after();
                    const int valid = min(kAtK, (own ? at_kend(a, w) : a.prefix_len) - key0), steps = (valid + 15) >> 4;
                    const uint64_t dv = at_desc_add(dv0, s * Sh::KB);
    #pragma unroll 1
                    for (int kk = 0; kk < steps; ++kk)       // O^T of the block alone
                        tc_mma_w(tmem + 64, at_desc_add(dv, kk * 16 * 128),
                                 at_desc_add(dp, (kk >> 2) * (kAtNarrow * 128) + (kk & 3) * 32), id_o, kk != 0);
                    tc_commit_w(smem_u32(o_full));
                    tc_commit_w(smem_u32(&kv_empty[s]));
                }
                blocks += w.nb;
            }
            tc_commit_w(smem_u32(done));
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kAnRegsSoftmax));
        AnCtx<D> c{&a, tid, ring, sp, s_full, p_full, o_full, x_full, x_empty, v_ragged, wmax, abort_flag, s_poison, tmem, 0, 0, 0, 0, 0};
        bool ok = !*abort_flag, more = true;
        AtWork w;
        for (int i = 0; ok; ++i) {
            if (!(ok = item(i, w, more)) || !more) break;
            const int rows = w.ntok * a.G;
            // The work on a block goes by the rows: 64 sequences of 3 tokens, 12 rows, over 600 keys take 47 us as 16 and 56
            // as 32; 512 single tokens of 4 rows over 200 keys 90 as 4, 94 as 8 and 102 as 16.
            ok = rows <= 4    ? an_item<D, 4>(c, w)
                 : rows <= 8  ? an_item<D, 8>(c, w)
                 : rows <= 16 ? an_item<D, 16>(c, w)
                              : an_item<D, 32>(c, w);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 5 && half == 0) {
        volatile int no_abort = 0;                   // every MMA of both halves has retired before the columns are freed
        mbar_wait(done, 0, &no_abort, nullptr);
        mbar_wait(reinterpret_cast<uint64_t*>(reinterpret_cast<unsigned char*>(done) + Sh::SMEM), 0, &no_abort, nullptr);
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, 256);
        tmem_relinquish();
    }
    pdl_wait();
}

// One warp per output row: m = max m_i, o = sum_i 2^(m_i - m) O_i / sum_i 2^(m_i - m) l_i
// over the row's own parts, then its prefix tile's, in their order. A part
// whose scores are all NaN has m = -inf as one that sees no key has, but a NaN
// in l; no part is left out of the sums, so that its NaN, or one that a weight
// of 0 meets in O, stays. Bound by
// the latency of its loads and by its own start, since no CTA of it fits beside
// those before it: lane i takes part i's m and l, and the first four parts'
// outputs are under way before these are there. Four CTAs per SM: decode of 64
// and of 256 behind a prefix 53 and 204 us; with three 55 and 205, with five 56
// and 212 (211 beside it), with eight 61 and 218. It ends 5 to 12 us after the
// kernel before it, for 5 to 17 MB read.
constexpr int kAtJoinCtas = 4;            // per SM
template <int D>
__global__ void __launch_bounds__(256, kAtJoinCtas) attn_combine_kernel(const RaggedAttnParams p) {
    constexpr int E = D / 32, AHEAD = 4;             // elements per lane, parts loaded together
    constexpr unsigned kAll = 0xffffffffu;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int G = p.hq_s / p.hkv_s, per = 2 * (kAtM / G), heads = p.N * p.hkv_s;
    // the lists are there when this kernel is launched (the kernels before it let it start once they have them), and are
    // read while those work; or the narrow kernel writes them
    if (p.few) pdl_wait();
    const unsigned units = (unsigned)__ldcg(&p.ctl->n_chunks) * heads;
    const int n_tok = __ldcg(&p.ctl->n_tokens);
    bool waited = p.few;
    for (unsigned u = blockIdx.x; u < units; u += gridDim.x) {
        const unsigned c = u / heads;
        const int h = u - c * heads, r = h / p.hkv_s;
        const int4 x0 = __ldcg(reinterpret_cast<const int4*>(p.chunks + c)), x1 = __ldcg(reinterpret_cast<const int4*>(p.chunks + c) + 1);
        const int t0 = x0.x, ntok = x0.y, qpos = x0.z, parts = x1.x;
        const int row = x1.y * 8 + warp;
        if (row >= ntok * G) continue;
        const int tok = row / G, g = row - tok * G, t = t0 + tok;
        const int64_t row0 = (int64_t)heads * G * t0 + (int64_t)h * ntok * G + row;
        const int64_t pos = (int64_t)qpos + tok;
        const int64_t stride = (int64_t)heads * ntok * G, first = x0.w + (int64_t)h * ntok * G + row - stride;
        int n2 = 0;
        int64_t row2 = 0, first2 = 0, stride2 = 0;
        if (p.shared) {
            const int i = t / per, k = min(per, n_tok - i * per);
            const int2 q = __ldcg(&p.prefix_groups[i]);
            n2 = q.y;
            stride2 = (int64_t)heads * k * G;
            const int64_t in_tile = (int64_t)h * k * G + (t - i * per) * G + g;
            row2 = (int64_t)heads * G * ((int64_t)p.T + i * per) + in_tile;
            first2 = q.x + in_tile - stride2;
        }
        const int n = parts + n2;
        auto at = [&](int i) {
            const int j = i - parts;
            return j < 0 ? (i ? first + i * stride : row0) : (j ? first2 + j * stride2 : row2);
        };
        if (!waited) {
            pdl_wait();
            waited = true;
        }
        float x[AHEAD][E];
        auto load = [&](int i0) {
#pragma unroll
            for (int i = 0; i < AHEAD; ++i) {
                if (i0 + i >= n) break;
                const float* src = p.part_o + at(i0 + i) * D + lane * E;
                if constexpr (E == 4) {
                    const float4 y = __ldcg(reinterpret_cast<const float4*>(src));
                    x[i][0] = y.x, x[i][1] = y.y, x[i][2] = y.z, x[i][3] = y.w;
                } else {
                    const float2 y = __ldcg(reinterpret_cast<const float2*>(src));
                    x[i][0] = y.x, x[i][1] = y.y;
                }
            }
        };
        load(0);
        float mx = -INFINITY;
        float2 ml = make_float2(-INFINITY, 0.f);     // lane's part of the first 32
        if (lane < n) ml = __ldcg(&p.part_ml[at(lane)]);
        mx = ml.x;
        for (int i = lane + 32; i < n; i += 32) mx = fmaxf(mx, p.part_ml[at(i)].x);
        mx = warp_max(mx);
        float f = 0.f, l = 0.f, o[E] = {};
        for (int i0 = 0; i0 < n; i0 += AHEAD) {
            if ((i0 & 31) == 0) {                    // weights of the next 32 parts
                if (i0) ml = i0 + lane < n ? p.part_ml[at(i0 + lane)] : make_float2(-INFINITY, 0.f);
                f = ml.x == -INFINITY ? 0.f : ex2_approx(ml.x - mx);
                l += warp_sum(f * ml.y);
            }
            if (i0) load(i0);
#pragma unroll
            for (int i = 0; i < AHEAD; ++i) {
                const float w = __shfl_sync(kAll, f, (i0 + i) & 31);
                if (i0 + i < n)
#pragma unroll
                    for (int k = 0; k < E; ++k) o[k] = fmaf(w, x[i][k], o[k]);
            }
        }
        const bool in = pos >= 0 && pos < p.max_kv;
        const float inv = 1.f / l;
        uint32_t y[E / 2];
#pragma unroll
        for (int k = 0; k < E / 2; ++k) y[k] = in ? pack_bf16x2(o[2 * k] * inv, o[2 * k + 1] * inv) : 0u;
        bf16* dst = static_cast<bf16*>(p.out) + (((int64_t)r * p.T + t) * p.hq_s + (h - r * p.hkv_s) * G + g) * D + lane * E;
        if constexpr (E == 4) *reinterpret_cast<uint2*>(dst) = make_uint2(y[0], y[1]);
        else *reinterpret_cast<uint32_t*>(dst) = y[0];
    }
    if (!waited) pdl_wait();
}

// ---------------------------------------------------------------------------
// launchers
// ---------------------------------------------------------------------------

namespace {
// 3-D bf16 map [d2][d1][d0], rows of d1 `stride1` elements apart and of d2 `stride2`; boxes b0 x b1 x b2, 128-byte swizzled.
cudaError_t attn_map(const void* base, int64_t d0, int64_t d1, int64_t d2, int64_t stride1, int64_t stride2, int b1, int b2,
                     CUtensorMap* out) {
    static std::mutex mu;
    static PFN_cuTensorMapEncodeTiled_v12000 encode = nullptr;
    {
        std::lock_guard<std::mutex> lock(mu);
        if (!encode) {
            cudaDriverEntryPointQueryResult q;
            cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", reinterpret_cast<void**>(&encode),
                                                             12000, cudaEnableDefault, &q);
            if (e != cudaSuccess || !encode) return e != cudaSuccess ? e : cudaErrorNotSupported;
        }
    }
    cuuint64_t gdim[3] = {(cuuint64_t)d0, (cuuint64_t)d1, (cuuint64_t)d2};
    cuuint64_t gstride[2] = {(cuuint64_t)stride1 * 2, (cuuint64_t)stride2 * 2};
    cuuint32_t box[3] = {64u, (cuuint32_t)b1, (cuuint32_t)b2};
    cuuint32_t estride[3] = {1u, 1u, 1u};
    CUresult r = encode(out, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), gdim, gstride, box, estride,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}
}  // namespace

AttnSizes attn_sizes(int64_t B, int64_t T, int hq, int hkv, int d) {
    const int64_t G = hq / hkv, per = 2 * (kAtM / G);
    // extra parts: their number times the target is at most all blocks
    const int64_t tiles = T / per + B + 1, prefix = T / per + 2, extra = 3 * kSMs / hkv + 2, extra_n = 5 * kSMs / hkv + 2;
    AttnSizes s;
    s.items = (size_t)(tiles + prefix + extra + extra_n + kSMs) * sizeof(AttnItem);
    s.prefix_groups = (size_t)prefix * sizeof(int2);
    s.chunks = (size_t)(T * G / 8 + tiles) * sizeof(AttnChunk);
    // every row once as a sequence's own and once as the prefix's, and the extra parts' rows
    const int64_t most = T < per ? T : per;
    s.rows = 2 * T * hq + extra * hkv * most * G + extra_n * hkv * (most * G < kAtNarrow ? most * G : kAtNarrow);
    s.part_ml = (size_t)s.rows * sizeof(float2);
    s.part_o = (size_t)s.rows * d * sizeof(float);
    return s;
}

cudaError_t launch_attn_plan(const RaggedAttnParams& p, cudaStream_t s) {
    RaggedAttnParams a = p;
    void* args[] = {&a};
    return launch_pdl(reinterpret_cast<const void*>(attn_plan_kernel), args, 1, 0, s, kPlanThreads);
}

cudaError_t launch_attn_ragged(const RaggedAttnParams& p, cudaStream_t s) {
    AtArgs a;
    memset(&a, 0, sizeof a);
    const int G = p.hq_s / p.hkv_s;
    a.N = p.N;
    a.T = p.T;
    a.hq_s = p.hq_s;
    a.hkv_s = p.hkv_s;
    a.G = G;
    a.tpt = kAtM / G;
    a.max_kv = p.max_kv;
    a.prefix_len = p.prefix_len;
    a.scale_log2 = p.scale_log2;
    a.status = p.status;
    a.out = static_cast<bf16*>(p.out);
    a.part_o = p.part_o;
    a.part_ml = p.part_ml;
    a.items = p.items;
    a.ctl = p.ctl;
    a.few = p.few;
    a.B = p.B;
    a.cu = p.cu;
    a.pos = p.pos;
    a.chunks = p.chunks;
    a.prefix_groups = p.prefix_groups;
    const int64_t D = p.d;
    cudaError_t e = attn_map(p.q, D, p.hq_s, (int64_t)p.N * p.T, D, p.hq_s * D, G, a.tpt, &a.tq);
    if (e == cudaSuccess) e = attn_map(p.q, D, p.hq_s, (int64_t)p.N * p.T, D, p.hq_s * D, G, kAtNarrow / G, &a.tqn);
    auto kv_maps = [&](int box) {                        // of both kernels, one after the other
        for (int r = 0; r < p.N && e == cudaSuccess; ++r) {
            a.v[r] = static_cast<const bf16*>(p.vc[r]);
            const int64_t groups = (int64_t)p.max_batch * p.hkv_s, rows = p.max_kv;
            e = attn_map(p.kc[r], D, rows, groups, D, rows * D, box, 1, &a.tk[r]);
            if (e == cudaSuccess) e = attn_map(p.vc[r], D, rows, groups, D, rows * D, box, 1, &a.tv[r]);
            if (p.prefix_len && e == cudaSuccess) {
                e = attn_map(p.pk[r], D, p.prefix_len, p.hkv_s, D, p.prefix_rows * D, box, 1, &a.pk[r]);
                if (e == cudaSuccess) e = attn_map(p.pv[r], D, p.prefix_len, p.hkv_s, D, p.prefix_rows * D, box, 1, &a.pv[r]);
            }
        }
    };
    if (e != cudaSuccess) return e;
    const bool d128 = p.d == 128;
    void* args[] = {&a};
    a.after_wide = p.T * (int64_t)G > p.narrow;          // else no item can have more rows
    if (a.after_wide) {
        const void* fn = d128 ? reinterpret_cast<const void*>(attn_items_kernel<128>)
                              : reinterpret_cast<const void*>(attn_items_kernel<64>);
        const int smem = d128 ? AtShape<128>::SMEM : AtShape<64>::SMEM;
        kv_maps(kAtK);
        if (e == cudaSuccess) e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e == cudaSuccess) e = launch_pdl(fn, args, kSMs, smem, s, kAtThreads);
        if (e != cudaSuccess) return e;
    }
    const void* fn = d128 ? reinterpret_cast<const void*>(attn_narrow_kernel<128>)
                          : reinterpret_cast<const void*>(attn_narrow_kernel<64>);
    const int smem = 2 * (d128 ? AnShape<128>::SMEM : AnShape<64>::SMEM) + (int)sizeof(AnFew);
    kv_maps(kAnBox);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e == cudaSuccess) e = launch_pdl(fn, args, kSMs, smem, s, kAnThreads);
    if (e != cudaSuccess) return e;
    RaggedAttnParams c = p;
    void* cargs[] = {&c};
    const int64_t units = ((int64_t)p.T * G / 8 + p.B) * p.N * p.hkv_s;
    return launch_pdl(d128 ? reinterpret_cast<const void*>(attn_combine_kernel<128>)
                           : reinterpret_cast<const void*>(attn_combine_kernel<64>),
                      cargs, (int)(units < kAtJoinCtas * kSMs ? units : kAtJoinCtas * kSMs), 0, s, 256);
}

}  // namespace tpk
