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
// Bound by memory for long calls (4096 rows of 14336 fp32 values 53 us, 5.5
// TB/s), by a workgroup's chain of load, maximum, barrier and store for short
// ones (2048 rows of 4096 bf16 values 10 us, twice its bytes' time).
#include <algorithm>

#include "i8.hpp"
#include "rows_i8.hpp"

namespace ttq {

template <bool F32, int SMODE, bool HOLD>
__global__ __launch_bounds__(1024) void k_quantize_rows(I8RowsArgs a) {
    quantize_rows<F32, SMODE, HOLD>(a, blockIdx.x, gridDim.x);
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
