// What the kernels around pages share: the check of a batch's offsets; which of
// the attention's two has a batch's sequences of few query rows.
#pragma once

#include "common.cuh"

namespace tpk {

// Whether the offsets of sequence b are not 0 = cu[0] <= cu[1] <= ... <= T. (Their difference is good behind this only: it can
// wrap around.)
__device__ __forceinline__ bool cu_bad(const int* cu, int b, int T) {
    const int from = cu[b], to = cu[b + 1];
    return to < from || from < 0 || to > T || (b == 0 && from != 0);
}

constexpr int kPnKeys = 32;               // keys of a chunk
constexpr int kPnRows = 16;               // query rows that a warp works on
constexpr int kPnMost = 32;               // ... of a sequence and KV head that are few, sixteen at a time
// Chunks of such sequences beside prompts that go with these: so few that their own kernel, which the prompts' has to wait
// for, would leave most of the machine idle. Single tokens behind 1000 keys and a prompt of 512, 8 KV heads of 128, with
// the prompt and apart: 8 tokens (2048 chunks) 37.1 and 43.1 us, 16 (4096) 42.7 and 45.9, 32 (8192) 62.6 and 51.6, 64 99.7
// and 65.7. Heads of 64: 33.1 and 39.1, 37.1 and 40.5, 53.1 and 44.2, 82.0 and 54.0. A prompt of 4096: 168.7 and 176.7, 178.1
// and 179.6, 194.9 and 185.4; of 128: 31.1 and 43.2, 36.9 and 45.9, 52.0 and 52.5. Behind 4000 keys (4032 chunks, 8064) 41.0
// and 46.3, 52.0 and 51.8; but 64 tokens behind 250 keys (4096 chunks) 60.0 and 47.9, since a head of a sequence costs the
// prompts' kernel three blocks besides its own, which a count of chunks does not see.
constexpr int64_t kPagedFewBeside = 5000;

// A head's query rows are worked on sixteen at a time.
__device__ __forceinline__ int paged_groups(int n, int G) { return (n * G + kPnRows - 1) / kPnRows; }
// Chunks of keys of a sequence (n new tokens from position pos on, pages for cap) for each head.
__device__ __forceinline__ int paged_chunks(int n, int pos, int cap) {
    const int64_t end = (int64_t)pos + n;
    const int kend = (int)(end < 0 ? 0 : end > cap ? cap : end);
    return max(1, (kend + kPnKeys - 1) / kPnKeys);
}
__device__ __forceinline__ int64_t paged_few_chunks(int n, int pos, int G, int cap) {
    return (int64_t)paged_chunks(n, pos, cap) * paged_groups(n, G);
}

}  // namespace tpk
