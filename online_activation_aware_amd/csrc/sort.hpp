// Tokens sorted by expert: a workgroup's part (sort.hip has the steps).
#pragma once

#include <algorithm>

#include "common.hpp"
#include "launch.hpp"

namespace ttq {

constexpr int kSortThreads = 1024, kSortWaves = kSortThreads / kWave;
constexpr int64_t kSortMaxBlocks = 256, kSortAlone = 2048;

// Slots per workgroup and workgroups for n slots.
static int64_t sort_span(int64_t n) {
    if (n <= kSortAlone) return kSortAlone;       // one launch
    const int64_t per = (n + kSortMaxBlocks - 1) / kSortMaxBlocks;
    return std::max<int64_t>((per + kSortThreads - 1) / kSortThreads, 1) * kSortThreads;
}
static int64_t sort_blocks(int64_t n) { return std::max<int64_t>((n + sort_span(n) - 1) / sort_span(n), 1); }

// The lanes whose key equals this lane's; `bits` bits of it count.
__device__ __forceinline__ uint64_t same_lanes(int key, int bits) {
    uint64_t m = ~0ull;
    for (int b = 0; b < bits; ++b) {
        const bool one = (key >> b) & 1;
        const uint64_t w = __ballot(one);
        m &= one ? w : ~w;
    }
    return m;
}

struct SortArgs {
    const int32_t* ids;
    int64_t n;
    int E, bits;                                  // bits of the keys 0 .. E
    int64_t span;
    int32_t *counts, *offsets, *order, *pos;      // counts [blocks][E] of each workgroup's slots
};

inline SortArgs sort_args(const int32_t* ids, int64_t n, int E, int32_t* offsets, int32_t* order, int32_t* pos,
                          int32_t* ws) {
    int bits = 1;
    while ((1 << bits) <= E) ++bits;
    return {ids, n, E, bits, sort_span(n), ws, offsets, order, pos};
}

// kSortThreads threads: the counts of slots [block * span, ...), or with PLACE
// their rows.
template <bool PLACE>
__device__ __forceinline__ void sort_block(const SortArgs& a, int block, int blocks) {
    const int32_t* __restrict__ ids = a.ids;
    const int64_t n = a.n, span = a.span;
    const int E = a.E, bits = a.bits;
    int32_t *counts = a.counts, *offsets = a.offsets, *order = a.order, *pos = a.pos;
    __shared__ int32_t place[kSortWaves][kMoeMaxExperts];
    __shared__ int32_t wsum[kSortWaves];
    const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
    const int64_t first = block * span;
    const int64_t w0 = first + wave * (span / kSortWaves), w1 = min(w0 + span / kSortWaves, n);
    for (int e = lane; e < E; e += kWave) place[wave][e] = 0;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    auto key_at = [&](int64_t i) __attribute__((always_inline)) {
        const int id = i < w1 ? ids[i] : -1;
        return id >= 0 && id < E ? id : E;        // E: no expert
    };
    // A wave alone touches its counts, and its LDS accesses are in order: between
    // its rounds only the compiler is held to that.
    for (int64_t i = w0; i < w1; i += kWave) {
        const int key = key_at(i + lane);
        const uint64_t m = same_lanes(key, bits);
        if (key < E && lane == __builtin_ctzll(m)) place[wave][key] += __builtin_popcountll(m);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    }
    __syncthreads();
    if constexpr (!PLACE) {
        for (int e = tid; e < E; e += kSortThreads) {
            int c = 0;
            for (int w = 0; w < kSortWaves; ++w) c += place[w][e];
            counts[(int64_t)block * E + e] = c;
        }
        return;
    }
    // Thread e: slots of expert e in all and before this workgroup, then the
    // experts' first rows by a scan over the threads.
    int all = 0, mine = 0;
    if (tid < E) {
        if (blocks == 1) {
            for (int w = 0; w < kSortWaves; ++w) all += place[w][tid];
        } else {
#pragma unroll 16
            for (int b = 0; b < blocks; ++b) {
                const int c = counts[b * E + tid];
                if (b < block) mine += c;
                all += c;
            }
        }
    }
    int sum = all;
#pragma unroll
    for (int s = 1; s < kWave; s <<= 1) {
        const int u = __shfl_up(sum, s);
        if (lane >= s) sum += u;
    }
    if (lane == kWave - 1) wsum[wave] = sum;
    __syncthreads();
    int before = 0, total = 0;
    for (int w = 0; w < kSortWaves; ++w) {
        if (w < wave) before += wsum[w];
        total += wsum[w];
    }
    if (tid < E) {
        const int lo = before + sum - all;
        if (block == 0) {
            offsets[tid] = lo;
            if (tid == 0) offsets[E] = total;
        }
        int at = lo + mine;
        for (int w = 0; w < kSortWaves; ++w) {
            const int c = place[w][tid];
            place[w][tid] = at;
            at += c;
        }
    }
    __syncthreads();
    for (int64_t i = w0; i < w1; i += kWave) {
        const int key = key_at(i + lane);
        const uint64_t m = same_lanes(key, bits);
        const int rank = __builtin_popcountll(m & ((1ull << lane) - 1));
        int r = -1;
        if (key < E) {
            r = place[wave][key] + rank;
            order[r] = (int32_t)(i + lane);
        }
        if (i + lane < w1) pos[i + lane] = r;
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        if (key < E && rank == 0) place[wave][key] += __builtin_popcountll(m);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    }
    // Behind the last row there is no slot.
    const int64_t end = min(first + span, n);
    for (int64_t r = max(first, (int64_t)total) + tid; r < end; r += kSortThreads) order[r] = -1;
}

}  // namespace ttq
