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

// A workgroup's tile where rows [offsets[e], offsets[e+1]) multiply matrix e: the
// rows [first, last) of its matrix and its tile of W.  first == last: none.
constexpr int kFewTiles = 96;                     // of an XCD: three for each of its compute units

struct I8Tile {
    int expert, first, last, mtile;
};

// Workgroups go to the eight XCDs in turn: an XCD has every eighth tile of each W
// (mt in all), so that all XCDs have the same work, and takes an expert's tiles of
// at most `size` rows one after the other for each of them, so that W comes from
// memory once.  Where the chip has few tiles a compute unit, the experts' last
// tiles of less than half the rows come behind all others instead (2048 tokens,
// two of eight experts, 14336 -> 4096: 350 us, 300 so).
//
// Every wave finds its own: the tiles of 64 experts at a time by a scan over the
// lanes.
__device__ __forceinline__ I8Tile find_tile(const int32_t* offsets, int E, int size, int mt, int block) {
    const int lane = threadIdx.x & (kWave - 1), per = (mt + 7) / 8, j = block / 8;
    int total = 0;
    for (int e0 = 0; e0 < E; e0 += kWave) {
        const int e = e0 + lane;
        int n = e < E ? (offsets[e + 1] - offsets[e] + size - 1) / size : 0;
#pragma unroll
        for (int s = 1; s < kWave; s <<= 1) n += __shfl_xor(n, s);
        total += __builtin_amdgcn_readfirstlane(n);
    }
    const int late = total * per <= kFewTiles ? size / 2 : 0;   // rows of tiles that come last
    int before = 0;                               // tiles of the experts before these 64
    for (int last = 0; last < (late ? 2 : 1); ++last)
        for (int e0 = 0; e0 < E; e0 += kWave) {
            const int e = e0 + lane;
            const int lo = e < E ? offsets[e] : 0, hi = e < E ? offsets[e + 1] : 0;
            const int first = late ? (hi - lo + late) / size : (hi - lo + size - 1) / size;   // tiles that come first
            const int nt = last ? (hi - lo > first * size) : first;
            int p = nt;
#pragma unroll
            for (int s = 1; s < kWave; s <<= 1) {
                const int u = __shfl_up(p, s);
                if (lane >= s) p += u;
            }
            const uint64_t who = __ballot((before + p) * per > j);
            if (who) {
                // (Read as scalars: a descriptor made of them is one for the wave.)
                const int l = __builtin_ctzll(who);
                auto at = [&](int x) { return __builtin_amdgcn_readlane(x, l); };
                const int n = at(nt), mine = j - (before + at(p) - n) * per, m = mine / n;
                const int row = at(lo) + ((last ? at(first) : 0) + mine - m * n) * size, mtile = block % 8 + 8 * m;
                return {e0 + l, row, mtile < mt ? min(row + size, at(hi)) : row, mtile};
            }
            before += __builtin_amdgcn_readlane(p, kWave - 1);
        }
    return {0, 0, 0, 0};
}

// Workgroups of find_tile: for an upper bound of the tiles of `size` rows.
inline int64_t i8_blocks(int64_t rows, int64_t E, int64_t size, int64_t mt) {
    const int64_t a = rows < E ? rows : E;
    return (a + (rows - a) / size) * ((mt + 7) / 8 * 8);
}

// The scale of output o's sum, or gate's, up's and s_down.
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

// 1 / s of four s_down within a unit of 2^-24, and whether all are far enough from
// the ends of fp32 for it.
struct I8Recip {
    f32x4 r;
    bool plain;
};
__device__ __forceinline__ I8Recip i8_recip(const f32x4& s) {
    I8Recip c;
    c.plain = true;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float r = __builtin_amdgcn_rcpf(s[i]);
        c.r[i] = __builtin_fmaf(__builtin_fmaf(-s[i], r, 1.f), r, r);
        c.plain &= __builtin_fabsf(s[i]) > 0x1p-100f && __builtin_fabsf(s[i]) < 0x1p100f;
    }
    return c;
}

// act(g) u / s, act(x) = x / (1 + exp(-y)), each operation rounded once (an h below
// 2^-100 perhaps a unit off): the quotients by corrected reciprocals, and by whole
// divisions where y, s or h is extreme.  An h that is off in its last bits has other
// codes next to borders: with exp2 of a rounded product and uncorrected reciprocals one
// result in 800 was another bf16 number.  (2048 tokens, two of eight experts, 4096 ->
// 14336: the layer 907 us, 29 more than with those; whole divisions alone take 55 more.)
__device__ __forceinline__ f32x4 i8_gate(const f32x4& g, const f32x4& u, const f32x4& s, const I8Recip& c, int act) {
    auto top = [](const f32x4& v) __attribute__((always_inline)) {
        return fmaxf(fmaxf(__builtin_fabsf(v[0]), __builtin_fabsf(v[1])), fmaxf(__builtin_fabsf(v[2]), __builtin_fabsf(v[3])));
    };
    f32x4 y = g, h;
    if (act != TTQ_ACT_SILU)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            y[i] = 1.5957691216057308f * (g[i] + 0.044715f * g[i] * g[i] * g[i]);   // 2 sqrt(2 / pi)
    bool plain = c.plain && top(y) < 87.f;
    if (plain) {
        f32x4 a;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float d = 1.f + expf(-y[i]), r = __builtin_amdgcn_rcpf(d);
            const float q = g[i] * r;
            a[i] = __builtin_fmaf(__builtin_fmaf(-q, d, g[i]), r, q) * u[i];
            h[i] = a[i] * c.r[i];
        }
        plain = top(h) < 0x1p127f;                // (a (1 / s) may be infinite where a / s is not)
#pragma unroll
        for (int i = 0; i < 4; ++i) h[i] = __builtin_fmaf(__builtin_fmaf(-h[i], s[i], a[i]), c.r[i], h[i]);
    }
    if (!plain)
#pragma unroll
        for (int i = 0; i < 4; ++i) h[i] = moe_act(g[i], act) * u[i] / s[i];
    return h;
}

// Results of four outputs: of the sums sg (and su, of gate and up).
template <bool GATE>
struct I8Results {
    f32x4 g, u, s;
    I8Recip c;
    __device__ __forceinline__ void set(int i, const I8Scales<GATE>& w) {
        g[i] = w.g;
        if constexpr (GATE) {
            u[i] = w.u;
            s[i] = w.s;
        }
    }
    __device__ __forceinline__ void ready() {     // all four are set
        if constexpr (GATE) c = i8_recip(s);
    }
    __device__ __forceinline__ f32x4 of(int act, float xs, const i32x4& sg, const i32x4& su) const {
        f32x4 y, v;
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = (float)sg[i] * xs * g[i];
        if constexpr (!GATE) return y;
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = (float)su[i] * xs * u[i];
        return i8_gate(y, v, s, c, act);
    }
};

}  // namespace ttq
