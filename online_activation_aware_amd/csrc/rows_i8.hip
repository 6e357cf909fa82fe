// Rows in 8 bits, symmetric, with one scale a row:
//   v = x, fp32(x s_j) or fp32(x / s_j);  a = max |v|;
//   scale = fp32(a / 127), 1 where that is 0;  q = clamp(rne(v / scale), -127, 127).
// A row with an infinity or NaN among its v gets the scale NaN and codes 0, so
// that every product of it is NaN and no other row's is touched.
//
// The code is the exact quotient's rounding, not that of a rounded quotient: q0 =
// rne(v r), r = fp32(1 / scale), is off by one only next to a border, and the
// remainder e = v - q0 scale, exact in one fma (a multiple of the smaller ulp,
// at most half a scale and a little), says on which side v lies.
//
// A workgroup takes whole rows: a lane holds two runs of eight values, read and
// written as whole vectors by consecutive lanes, and the row's maximum is that
// of the bit patterns (a NaN is above every number).  Rows of more than 16384
// values are read twice, the second time from the cache.
#include <algorithm>

#include "i8.hpp"
#include "wave.hpp"

namespace ttq {

constexpr int kRowSeg = 8;                        // values of a vector
constexpr int kRowSegs = 2;                       // vectors a lane holds

template <bool F32>
__device__ __forceinline__ void load8(const void* X, int64_t at, float (&f)[kRowSeg]) {
    if constexpr (F32) {
        const f32x4 a = *(const f32x4*)((const float*)X + at), b = *(const f32x4*)((const float*)X + at + 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[i] = a[i];
            f[4 + i] = b[i];
        }
    } else {
        const u32x4 u = *(const u32x4*)((const uint16_t*)X + at);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = bf16lo_to_f32(u[i]);
            f[2 * i + 1] = bf16hi_to_f32(u[i]);
        }
    }
}

__device__ __forceinline__ uint32_t pack4(const int (&q)[4]) {
    return (q[0] & 0xFF) | (q[1] & 0xFF) << 8 | (q[2] & 0xFF) << 16 | (uint32_t)q[3] << 24;
}

// rne(v / scale) of the exact quotient, |v| <= 127.5 scale or so.
__device__ __forceinline__ float code_of(float v, float scale, float r) {
    float q = __builtin_rintf(v * r);
    const float e = __builtin_fmaf(-q, scale, v), d = 2.f * __builtin_fabsf(e);
    const bool odd = ((int)q & 1) != 0;
    if (d > scale || (d == scale && odd)) q += __builtin_copysignf(1.f, e);
    return fminf(fmaxf(q, -127.f), 127.f);
}
// The same where 1 / scale overflows or e could be rounded: in 64 bits the
// quotient of two 24-bit numbers lands on a border only if it is one.
__device__ __forceinline__ float code_of_tiny(float v, float scale) {
    return fminf(fmaxf((float)__builtin_rint((double)v / (double)scale), -127.f), 127.f);
}

template <bool F32, int SMODE, bool HOLD>
__global__ __launch_bounds__(1024) void k_quantize_rows(I8RowsArgs a) {
    __shared__ uint32_t part[16];
    const int tid = threadIdx.x, nt = blockDim.x, nw = nt / kWave;
    const int64_t R = a.nrows ? *a.nrows : a.R;
    const int runs = (int)((a.K + (int64_t)nt * kRowSeg - 1) / ((int64_t)nt * kRowSeg));
    for (int64_t r = blockIdx.x; r < R; r += gridDim.x) {
        const int slot = a.order ? a.order[r] : 0;
        const int64_t src = a.order ? slot / a.topk : r;
        const float* s = SMODE ? a.s + (a.ids ? (int64_t)a.ids[slot] * a.s_stride : 0) : nullptr;
        float v[kRowSegs][kRowSeg];
        auto value = [&](int64_t k, float (&f)[kRowSeg]) __attribute__((always_inline)) {
            load8<F32>(a.X, src * a.ldx + k, f);
            if constexpr (SMODE) {
                float sf[kRowSeg];
                load8<true>(s, k, sf);
#pragma unroll
                for (int i = 0; i < kRowSeg; ++i) f[i] = SMODE == 1 ? f[i] * sf[i] : f[i] / sf[i];
            }
        };
        uint32_t top = 0;
        auto highest = [&](const float (&f)[kRowSeg]) __attribute__((always_inline)) {
#pragma unroll
            for (int i = 0; i < kRowSeg; ++i) top = max(top, __builtin_bit_cast(uint32_t, f[i]) & 0x7FFFFFFFu);
        };
        if constexpr (HOLD) {
#pragma unroll
            for (int u = 0; u < kRowSegs; ++u) {
                const int64_t k = ((int64_t)u * nt + tid) * kRowSeg;
                if (k < a.K) value(k, v[u]);
                else
#pragma unroll
                    for (int i = 0; i < kRowSeg; ++i) v[u][i] = 0.f;
                highest(v[u]);
            }
        } else {
            for (int u = 0; u < runs; ++u) {
                const int64_t k = ((int64_t)u * nt + tid) * kRowSeg;
                if (k >= a.K) break;
                value(k, v[0]);
                highest(v[0]);
            }
        }
        top = wave_max_u32(top);
        if (nw > 1) {
            if ((tid & (kWave - 1)) == 0) part[tid / kWave] = top;
            __syncthreads();
            for (int w = 0; w < nw; ++w) top = max(top, part[w]);
            __syncthreads();
        }
        const bool bad = top >= 0x7F800000u;      // an infinity or NaN
        float scale = __builtin_bit_cast(float, top) / 127.f;
        if (scale == 0.f) scale = 1.f;
        if (bad) scale = __builtin_nanf("");
        if (tid == 0) a.scale[r] = scale;
        const float rs = 1.f / scale;
        const bool tiny = scale < 0x1p-100f;
        auto store = [&](int64_t k, const float (&f)[kRowSeg]) __attribute__((always_inline)) {
            int q[kRowSeg];
#pragma unroll
            for (int i = 0; i < kRowSeg; ++i)
                q[i] = bad ? 0 : (int)(tiny ? code_of_tiny(f[i], scale) : code_of(f[i], scale, rs));
            u32x2 p;
#pragma unroll
            for (int h = 0; h < 2; ++h) p[h] = pack4({q[4 * h], q[4 * h + 1], q[4 * h + 2], q[4 * h + 3]});
            *(u32x2*)(a.codes + r * a.ldc + k) = p;
        };
        if constexpr (HOLD) {
#pragma unroll
            for (int u = 0; u < kRowSegs; ++u) {
                const int64_t k = ((int64_t)u * nt + tid) * kRowSeg;
                if (k < a.K) store(k, v[u]);
            }
        } else {
            for (int u = 0; u < runs; ++u) {
                const int64_t k = ((int64_t)u * nt + tid) * kRowSeg;
                if (k >= a.K) break;
                value(k, v[0]);
                store(k, v[0]);
            }
        }
    }
}

hipError_t launch_quantize_rows(const I8RowsArgs& a, hipStream_t st) {
    const int64_t lanes = (a.K + kRowSeg * kRowSegs - 1) / (kRowSeg * kRowSegs);
    const int nt = (int)std::min<int64_t>((lanes + kWave - 1) / kWave * kWave, 1024);
    const bool hold = lanes <= 1024;
    // Rows are taken in turn by at most eight rounds of the workgroups that fit.
    const dim3 grid((unsigned)std::min<int64_t>(a.R, 256 * 2048 / nt * 8)), block((unsigned)nt);
    const int mode = a.s == nullptr ? 0 : a.divide ? 2 : 1;
#define TTQ_R3(F, S, H) return launch_kernel(k_quantize_rows<F, S, H>, grid, block, 0, st, nullptr, nullptr, a)
#define TTQ_R2(F, S)          \
    do {                      \
        if (hold) TTQ_R3(F, S, true); \
        TTQ_R3(F, S, false);  \
    } while (0)
#define TTQ_R1(F)                  \
    do {                           \
        if (mode == 0) TTQ_R2(F, 0); \
        if (mode == 1) TTQ_R2(F, 1); \
        TTQ_R2(F, 2);              \
    } while (0)
    if (a.xf32) TTQ_R1(true);
    TTQ_R1(false);
#undef TTQ_R1
#undef TTQ_R2
#undef TTQ_R3
}

}  // namespace ttq
