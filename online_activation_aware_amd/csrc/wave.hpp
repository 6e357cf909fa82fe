// Reductions over a wave by DPP (a lane exchange through LDS costs a hundred
// cycles a step).
#pragma once

#include "common.hpp"

namespace ttq {

// Combine over the wave by DPP: rows of 16 lanes by shifts, then the rows;
// lane 63 holds the result.  `none`: the value of lanes that have no partner.
template <typename F>
__device__ __forceinline__ uint32_t wave_combine(uint32_t v, uint32_t none, F f) {
#define TTQ_DPP(ctrl, rows) v = f(v, (uint32_t)__builtin_amdgcn_update_dpp((int)none, (int)v, ctrl, rows, 0xF, false))
    TTQ_DPP(0x111, 0xF);   // row_shr 1, 2, 4, 8
    TTQ_DPP(0x112, 0xF);
    TTQ_DPP(0x114, 0xF);
    TTQ_DPP(0x118, 0xF);
    TTQ_DPP(0x142, 0xA);   // row_bcast 15 into rows 1 and 3
    TTQ_DPP(0x143, 0xC);   // row_bcast 31 into rows 2 and 3
#undef TTQ_DPP
    return (uint32_t)__builtin_amdgcn_readlane((int)v, kWave - 1);
}
__device__ __forceinline__ float wave_sum(float x) {
    return __builtin_bit_cast(float, wave_combine(__builtin_bit_cast(uint32_t, x), 0u, [](uint32_t a, uint32_t b) {
        return __builtin_bit_cast(uint32_t, __builtin_bit_cast(float, a) + __builtin_bit_cast(float, b));
    }));
}
__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v) {
    return wave_combine(v, 0u, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
}

}  // namespace ttq
