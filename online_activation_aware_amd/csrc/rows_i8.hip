// Rows in 8 bits, symmetric, with one scale a row:
//   v = x, fp32(x s_j) or fp32(x / s_j);  a = max |v|;
//   scale = fp32(a / 127), 1 where that is 0;  q = clamp(rne(v / scale), -127, 127).
// A row with an infinity or NaN among its v gets the scale NaN and codes 0, so
// that every product of it is NaN and no other row's is touched.
//
// The code is the exact quotient's rounding, not that of a rounded quotient: q =
// rne(v r), r = fp32(1 / scale), is off by one only next to a border, and the
// remainder e = v - q scale, exact in one fma (a multiple of the smaller ulp,
// at most half a scale and a little), says on which side v lies.  v = x / s is
// the IEEE quotient from fp32(1 / s) by two corrections (as in Markstein, "IA-64
// and Elementary Functions", 2000), where no exponent is extreme.
//
// A workgroup takes whole rows, one after the other, the next one's values
// requested before the work on this one: a lane holds two runs of eight values,
// read and written as whole vectors by consecutive lanes, and its s and 1 / s;
// the row's maximum is that of the bit patterns (a NaN is above every number).
// Rows of more than 16384 values are read twice, the second time from the cache.
#include <algorithm>

#include "i8.hpp"
#include "rows_i8.hpp"
#include "wave.hpp"

namespace ttq {

constexpr int kRowSegs = 2;                       // vectors a lane holds

template <bool F32, int SMODE, bool HOLD>
__global__ __launch_bounds__(1024) void k_quantize_rows(I8RowsArgs a) {
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
    if (HOLD && blockIdx.x < R) request(blockIdx.x);
    int turn = 0;
    for (int64_t r = blockIdx.x; r < R; r += gridDim.x, turn ^= 1) {
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
            if (r + gridDim.x < R && !a.ids) request(r + gridDim.x);
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
        if (SMODE == 2 && top < kRowTiny) {       // quotients near the lowest exponents
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
            if (r + gridDim.x < R && a.ids) request(r + gridDim.x);
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

hipError_t launch_quantize_rows(const I8RowsArgs& a, hipStream_t st) {
    const int64_t lanes = (a.K + kRowSeg * kRowSegs - 1) / (kRowSeg * kRowSegs);
    const int nt = (int)std::min<int64_t>((lanes + kWave - 1) / kWave * kWave, 1024);
    const bool hold = lanes <= 1024;
    // As many workgroups as fit the chip at 1024 lanes a compute unit.
    const dim3 grid((unsigned)std::min<int64_t>(a.R, 256 * (1024 / nt))), block((unsigned)nt);
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
