// Linear layers in 8-bit integers: what their kernels share.
#pragma once

#include "common.hpp"
#include "launch.hpp"
#include "lds_dma.hpp"
#include "moe.hpp"

namespace ttq {

typedef __attribute__((__vector_size__(4 * sizeof(int)))) int i32x4;

// Up to 16 x 16 sums of 64 channels each, exact in int32.
__device__ __forceinline__ i32x4 mfma_i8(const u32x4& a, const u32x4& b, const i32x4& c) {
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, a), __builtin_bit_cast(i32x4, b), c, 0, 0, 0);
}

// The matrix of a tile of rows and the rows of it: [first, last).
struct I8Tile {
    int expert;
    int64_t first, last;
};

// Tile `tile` of at most `size` rows each, where rows [offsets[e], offsets[e+1])
// multiply matrix e (offsets null: all rows matrix 0); first == last where
// there are fewer.  Every wave finds its own: the tiles of 64 experts at a
// time by a scan over the lanes.
__device__ __forceinline__ I8Tile find_tile(const int32_t* offsets, int E, int64_t rows, int size, int64_t tile) {
    if (offsets == nullptr) {
        const int64_t f = tile * size;
        return {0, f < rows ? f : rows, f + size < rows ? f + size : rows};
    }
    const int lane = threadIdx.x & (kWave - 1);
    int64_t before = 0;                           // tiles of the experts before these 64
    for (int e0 = 0; e0 < E; e0 += kWave) {
        const int e = e0 + lane;
        const int lo = e < E ? offsets[e] : 0, hi = e < E ? offsets[e + 1] : 0;
        const int nt = (hi - lo + size - 1) / size;
        int p = nt;
#pragma unroll
        for (int s = 1; s < kWave; s <<= 1) {
            const int u = __shfl_up(p, s);
            if (lane >= s) p += u;
        }
        const uint64_t who = __ballot(before + p > tile);
        if (who) {
            const int l = __builtin_ctzll(who);
            const int64_t first = __shfl(lo, l) + (tile - before - (__shfl(p, l) - __shfl(nt, l))) * size;
            const int64_t end = __shfl(hi, l);
            return {e0 + l, first, first + size < end ? first + size : end};
        }
        before += __shfl(p, kWave - 1);
    }
    return {0, 0, 0};
}

// Upper bound of the tiles of `size` rows over E experts.
inline int64_t i8_tiles(int64_t rows, int64_t E, int64_t size) {
    const int64_t a = rows < E ? rows : E;
    return a + (rows - a) / size;
}

// A result of the sums s (of gate and up: sg and su).
template <bool GATE>
__device__ __forceinline__ float i8_result(const I8Product& p, int expert, int64_t o, float xs, int sg, int su) {
    const float* ws = p.w_scale + expert * p.M * (GATE ? 2 : 1);
    const float g = (float)sg * xs * ws[o];
    if constexpr (!GATE) return g;
    const float u = (float)su * xs * ws[p.M + o];
    return moe_act(g, p.act) * u / p.s_down[expert * p.s_stride + o];
}

}  // namespace ttq
