// Rows in 8 bits: a lane's and a workgroup's part (rows_i8.hip has the mathematics).
#pragma once

#include "common.hpp"
#include "launch.hpp"
#include "wave.hpp"

namespace ttq {

constexpr int kRowSeg = 8;                        // values of a vector
constexpr uint32_t kRowTiny = 0x24800000u;        // 2^-54
constexpr uint32_t kRowHuge = 0x7F000000u;        // 2^127

// Eight values of a row as they lie in memory.
template <bool F32>
struct RowVector {
    u32x4 w[F32 ? 2 : 1];
    __device__ __forceinline__ void load(const void* X, int64_t at) {
        const u32x4* p = (const u32x4*)((const char*)X + at * (F32 ? 4 : 2));
        w[0] = p[0];
        if constexpr (F32) w[1] = p[1];
    }
    __device__ __forceinline__ float operator[](int i) const {
        const uint32_t u = w[F32 ? i / 4 : 0][F32 ? i % 4 : i / 2];   // (a copy: a bit cast of the element takes the first)
        if constexpr (F32) return __builtin_bit_cast(float, u);
        return i % 2 ? bf16hi_to_f32(u) : bf16lo_to_f32(u);
    }
};

// The eight channels' scales: none (MODE 0), factors (1) or divisors (2).
template <int MODE>
struct RowScale {
    float s[MODE ? kRowSeg : 1], r[MODE == 2 ? kRowSeg : 1];
    bool plain;                                   // no exponent of s is extreme
    __device__ __forceinline__ void load(const float* p) {
        if constexpr (MODE) {
            const f32x4 a = *(const f32x4*)p, b = *(const f32x4*)(p + 4);
#pragma unroll
            for (int i = 0; i < kRowSeg; ++i) s[i] = i < 4 ? a[i] : b[i - 4];
        }
        if constexpr (MODE == 2) {
            plain = true;
#pragma unroll
            for (int i = 0; i < kRowSeg; ++i) {
                r[i] = 1.f / s[i];
                plain &= __builtin_fabsf(s[i]) > 0x1p-40f && __builtin_fabsf(s[i]) < 0x1p40f;
            }
        }
    }
};

// v of the eight values: x, fp32(x s) or fp32(x / s).  exact: by the division
// itself, for rows whose quotients are near the largest number (x (1 / s) may be
// beyond it where x / s is not) or tiny: x - q s has no bit below fp32's last, 2^-149,
// where |s| > 2^-40 and q >= 2^-63, and in a row whose largest quotient is 2^-54 or more the
// codes of smaller ones are 0.
template <bool F32, int MODE>
__device__ __forceinline__ void row_values(const RowVector<F32>& x, const RowScale<MODE>& s, bool exact,
                                           float (&v)[kRowSeg]) {
    if constexpr (MODE == 2) {
        if (exact || !s.plain) {
#pragma unroll
            for (int i = 0; i < kRowSeg; ++i) v[i] = x[i] / s.s[i];
            return;
        }
#pragma unroll
        for (int i = 0; i < kRowSeg; ++i) {
            float q = x[i] * s.r[i];
            q = __builtin_fmaf(__builtin_fmaf(-q, s.s[i], x[i]), s.r[i], q);
            v[i] = __builtin_fmaf(__builtin_fmaf(-q, s.s[i], x[i]), s.r[i], q);
        }
    } else {
#pragma unroll
        for (int i = 0; i < kRowSeg; ++i) v[i] = MODE == 1 ? x[i] * s.s[i] : x[i];
    }
}

__device__ __forceinline__ uint32_t row_top(const float (&v)[kRowSeg], uint32_t top) {
#pragma unroll
    for (int i = 0; i < kRowSeg; ++i) top = max(top, __builtin_bit_cast(uint32_t, v[i]) & 0x7FFFFFFFu);
    return top;
}

// The scale of a row whose largest |v| has these bits.
__device__ __forceinline__ float row_scale(uint32_t top) {
    if (top >= 0x7F800000u) return __builtin_nanf("");
    const float scale = __builtin_bit_cast(float, top) / 127.f;
    return scale == 0.f ? 1.f : scale;
}

// The codes of eight values; 0 for a row whose scale is NaN.
__device__ __forceinline__ u32x2 row_codes(const float (&v)[kRowSeg], float scale) {
    constexpr float kMagic = 12582912.f;          // 1.5 2^23: a sum with it is a whole number, its low byte the code
    uint32_t b[kRowSeg];
    if (!(scale >= 0x1p-100f)) {
        // 1 / scale could overflow, the remainder be rounded, the scale lie well
        // below a / 127: in 64 bits the quotient of two 24-bit numbers lands on a
        // border only if it is one.
#pragma unroll
        for (int i = 0; i < kRowSeg; ++i) {
            const double q = __builtin_rint((double)v[i] / (double)scale);
            b[i] = scale == scale ? (uint32_t)(int)fmin(fmax(q, -127.0), 127.0) : 0u;
        }
    } else {
        const float r = 1.f / scale, half = 0.5f * scale;
        float t[kRowSeg];
        bool off = false;
#pragma unroll
        for (int i = 0; i < kRowSeg; ++i) {
            t[i] = __builtin_fmaf(v[i], r, kMagic);
            off |= !(__builtin_fabsf(__builtin_fmaf(-(t[i] - kMagic), scale, v[i])) < half);
        }
        if (off) {                                // a value on a border or on its wrong side
#pragma unroll
            for (int i = 0; i < kRowSeg; ++i) {
                const float e = __builtin_fmaf(-(t[i] - kMagic), scale, v[i]), d = __builtin_fabsf(e);
                const bool odd = __builtin_bit_cast(uint32_t, t[i]) & 1u;
                if (d > half || (d == half && odd)) t[i] += __builtin_copysignf(1.f, e);
            }
        }
#pragma unroll
        for (int i = 0; i < kRowSeg; ++i) b[i] = __builtin_bit_cast(uint32_t, t[i]);
    }
    u32x2 p;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint32_t lo = __builtin_amdgcn_perm(b[4 * h + 1], b[4 * h], 0x0C0C0400u);
        const uint32_t hi = __builtin_amdgcn_perm(b[4 * h + 3], b[4 * h + 2], 0x04000C0Cu);
        p[h] = lo | hi;
    }
    return p;
}

constexpr int kRowSegs = 2;                       // vectors a lane holds

// The whole rows `block`, block + blocks, ... by a workgroup (HOLD: of at most 16
// values a lane).
template <bool F32, int SMODE, bool HOLD>
__device__ __forceinline__ void quantize_rows(const I8RowsArgs& a, int block, int blocks) {
    constexpr int S = HOLD ? kRowSegs : 1;
    __shared__ uint32_t part[2][16];
    const int tid = threadIdx.x, nt = blockDim.x, nw = nt / kWave;
    const int64_t R = a.nrows ? *a.nrows : a.R;
    const int K = (int)a.K, runs = (K + nt * kRowSeg - 1) / (nt * kRowSeg);
    RowScale<SMODE> s[S];
    RowVector<F32> next[S];
    auto source = [&](int64_t r, int& slot) __attribute__((always_inline)) {
        slot = a.order ? a.order[r] : 0;
        return a.order ? slot / a.topk : r;
    };
    auto request = [&](int64_t r) __attribute__((always_inline)) {
        int slot;
        const int64_t src = source(r, slot);
#pragma unroll
        for (int u = 0; u < S; ++u) {
            const int k = (u * nt + tid) * kRowSeg;
            if (k < K) {
                next[u].load(a.X, src * a.ldx + k);
                if (a.ids) s[u].load(a.s + (int64_t)a.ids[slot] * a.s_stride + k);
            }
        }
    };
    if (HOLD && !a.ids)
#pragma unroll
        for (int u = 0; u < S; ++u) {
            const int k = (u * nt + tid) * kRowSeg;
            if (k < K) s[u].load(a.s + k);
        }
    if (HOLD && block < R) request(block);
    int turn = 0;
    for (int64_t r = block; r < R; r += blocks, turn ^= 1) {
        float v[S][kRowSeg] = {};
        uint32_t top = 0;
        int slot;
        const int64_t src = source(r, slot);
        // (Rows read twice: run u's values into v[0].)
        auto value = [&](int k, bool exact) __attribute__((always_inline)) {
            RowVector<F32> x;
            x.load(a.X, src * a.ldx + k);
            s[0].load(a.s + (a.ids ? (int64_t)a.ids[slot] * a.s_stride : 0) + k);
            row_values(x, s[0], exact, v[0]);
        };
        RowVector<F32> x[S];
        if constexpr (HOLD) {
#pragma unroll
            for (int u = 0; u < S; ++u) {
                x[u] = next[u];
                if ((u * nt + tid) * kRowSeg < K) row_values(x[u], s[u], false, v[u]);
                top = row_top(v[u], top);
            }
            if (r + blocks < R && !a.ids) request(r + blocks);
        } else {
            for (int u = 0; u < runs; ++u) {
                const int k = (u * nt + tid) * kRowSeg;
                if (k >= K) break;
                value(k, false);
                top = row_top(v[0], top);
            }
        }
        auto whole = [&](int half) __attribute__((always_inline)) {   // of the row
            top = wave_max_u32(top);
            if (nw > 1) {
                // (Turns alternate between two arrays: one barrier a turn.)
                if ((tid & (kWave - 1)) == 0) part[half][tid / kWave] = top;
                __syncthreads();
                for (int w = 0; w < nw; ++w) top = max(top, part[half][w]);
            }
        };
        whole(turn);
        bool exact = false;
        if (SMODE == 2 && (top < kRowTiny || top >= kRowHuge)) {   // quotients near the ends of fp32
            exact = true;
            __syncthreads();
            top = 0;
            if constexpr (HOLD) {
#pragma unroll
                for (int u = 0; u < S; ++u) {
                    if ((u * nt + tid) * kRowSeg < K) row_values(x[u], s[u], true, v[u]);
                    top = row_top(v[u], top);
                }
            } else {
                for (int u = 0; u < runs; ++u) {
                    const int k = (u * nt + tid) * kRowSeg;
                    if (k >= K) break;
                    value(k, true);
                    top = row_top(v[0], top);
                }
            }
            whole(turn);
            __syncthreads();
        }
        const float scale = row_scale(top);
        if (tid == 0) a.scale[r] = scale;
        if constexpr (HOLD) {
#pragma unroll
            for (int u = 0; u < S; ++u) {
                const int k = (u * nt + tid) * kRowSeg;
                if (k < K) *(u32x2*)(a.codes + r * a.ldc + k) = row_codes(v[u], scale);
            }
            if (r + blocks < R && a.ids) request(r + blocks);
        } else {
            for (int u = 0; u < runs; ++u) {
                const int k = (u * nt + tid) * kRowSeg;
                if (k >= K) break;
                value(k, exact);
                *(u32x2*)(a.codes + r * a.ldc + k) = row_codes(v[0], scale);
            }
        }
    }
}

}  // namespace ttq
