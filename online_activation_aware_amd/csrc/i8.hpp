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
    int first, last;
};

// Tile `tile` of at most `size` rows each, where rows [offsets[e], offsets[e+1])
// multiply matrix e (offsets null: all rows matrix 0); first == last where
// there are fewer.  Every wave finds its own: the tiles of 64 experts at a
// time by a scan over the lanes.
__device__ __forceinline__ I8Tile find_tile(const int32_t* offsets, int E, int rows, int size, int tile) {
    if (offsets == nullptr) {
        const int f = min(tile * size, rows);
        return {0, f, min(f + size, rows)};
    }
    const int lane = threadIdx.x & (kWave - 1);
    int before = 0;                               // tiles of the experts before these 64
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
            // (Read as scalars: a descriptor made of them is one for the wave.)
            const int l = __builtin_ctzll(who);
            auto at = [&](int x) { return __builtin_amdgcn_readlane(x, l); };
            const int first = at(lo) + (tile - before - (at(p) - at(nt))) * size;
            return {e0 + l, first, min(first + size, at(hi))};
        }
        before += __builtin_amdgcn_readlane(p, kWave - 1);
    }
    return {0, 0, 0};
}

// Upper bound of the tiles of `size` rows over E experts.
inline int64_t i8_tiles(int64_t rows, int64_t E, int64_t size) {
    const int64_t a = rows < E ? rows : E;
    return a + (rows - a) / size;
}

// The scales of output o: of its sum, or of gate's and up's and 1 / s_down's s.
template <bool GATE>
struct I8Scales {
    float g, u, s;
};
template <bool GATE>
__device__ __forceinline__ I8Scales<GATE> i8_scales(const I8Product& p, int expert, int64_t o) {
    const float* ws = p.w_scale + expert * p.M * (GATE ? 2 : 1);
    if constexpr (GATE) return {ws[o], ws[p.M + o], p.s_down[expert * p.s_stride + o]};
    return {ws[o], 0.f, 0.f};
}

// A result of the sums sg (and su, of gate and up).
template <bool GATE>
__device__ __forceinline__ float i8_result(const I8Scales<GATE>& w, int act, float xs, int sg, int su) {
    const float g = (float)sg * xs * w.g;
    if constexpr (!GATE) return g;
    const float u = (float)su * xs * w.u;
    return moe_act(g, act) * u / w.s;
}

}  // namespace ttq
