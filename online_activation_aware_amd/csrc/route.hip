// Router of a mixture-of-experts layer: each token's top-k experts and their
// weights from its logits.
//
//   ids[t][j]: the experts of the j-th largest logit, ties to the lowest
//   index; softmax: w = exp(l_j - m) / sum_e exp(l_e - m), m the row's
//   maximum; sigmoid: w = 1 / (1 + exp(-l_j)); renormalised: w / sum_j w.  A
//   sigmoid of l < 0 is exp(l) / (1 + exp(l)); to be renormalised, of exp(l - m),
//   so that the ratios of scores below fp32's range are kept.
//
// One wave per token: lane l holds the logits l, l + 64, ... as 32-bit keys
// that order like the floats (NaN and -inf as the key 0, which is never
// chosen).  k rounds pick the experts: the wave's largest key by DPP (a lane
// exchange through LDS would cost a hundred cycles a step: 8192 tokens of 160
// bf16 logits, 6 experts each, 10.7 us so and 6.7 us now), the lowest index that
// has it by ballots; its lane retires it.  The sum of the softmax comes from
// the same registers, in fp32 and in a fixed order.  The pass reads the logits
// once; a call is bound by its launch and the rounds' dependent steps.
#include "common.hpp"
#include "launch.hpp"

namespace ttq {

constexpr int kRouteWaves = 4;                    // tokens per workgroup

__device__ __forceinline__ uint32_t order_key(float x) {
    if (!(x > -__builtin_inff())) return 0u;      // -inf and NaN
    const uint32_t b = __builtin_bit_cast(uint32_t, x + 0.0f);   // -0 equals +0
    return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
    return __builtin_bit_cast(float, (k & 0x80000000u) ? k ^ 0x80000000u : ~k);
}
// exp(v - m) with exp(m - m) = 1 for an infinite m.
__device__ __forceinline__ float exp_below(float v, float m) { return v == m ? 1.f : expf(v - m); }

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

template <int NV, bool LF32>
__global__ __launch_bounds__(kRouteWaves * kWave) void k_moe_route(const void* __restrict__ L, int64_t T, int E,
                                                                   int64_t ldl, int topk, int score, int renorm,
                                                                   int32_t* __restrict__ ids,
                                                                   float* __restrict__ wts) {
    const int lane = threadIdx.x & (kWave - 1);
    const int64_t t = (int64_t)blockIdx.x * kRouteWaves + threadIdx.x / kWave;
    if (t >= T) return;
    uint32_t key[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int e = lane + kWave * i;
        float v = -__builtin_inff();
        if (e < E) {
            if constexpr (LF32) v = ((const float*)L)[t * ldl + e];
            else v = bf16_to_f32(((const uint16_t*)L)[t * ldl + e]);
        }
        key[i] = order_key(v);
    }
    uint32_t mine = 0, mine_id = 0xFFFFFFFFu;     // the lane-th choice
    float m = 0.f, sum = 1.f;
    uint32_t taken = 0;                           // bit i: this lane's value i is chosen already
    for (int j = 0; j < topk; ++j) {
        uint32_t bk = 0;
        int bi = 0;                               // this lane's best value left, the lowest of equals
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const bool better = key[i] > bk && !((taken >> i) & 1u);
            bk = better ? key[i] : bk;
            bi = better ? i : bi;
        }
        const uint32_t top = wave_combine(bk, 0u, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
        if (top == 0) break;                      // nothing is left to choose
        uint64_t who = 0;
        int i = 0;
        for (; i < NV; ++i) {                     // expert lane + 64 i: the lowest i first
            who = __ballot(bk == top && bi == i);
            if (who) break;
        }
        const int owner = __builtin_ctzll(who);
        if (lane == owner) taken |= 1u << i;
        bk = top;
        const uint32_t be = (uint32_t)(owner + kWave * i);
        if (lane == j) {
            mine = bk;
            mine_id = be;
        }
        if (j == 0) m = key_value(bk);
    }
    if (score == TTQ_SCORE_SOFTMAX) {
        float part = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) part += key[i] ? exp_below(key_value(key[i]), m) : 0.f;
        sum = wave_sum(part);
    }
    // Below -745 the scores are none in 64 bits either (rows masked by a lowest
    // finite value): they stay 0.
    const float base = renorm && m < 0.f && m >= -745.f ? m : 0.f;
    float w = 0.f;
    if (mine) {
        const float v = key_value(mine);
        if (score == TTQ_SCORE_SOFTMAX) w = exp_below(v, m) / sum;
        else w = v < 0.f ? expf(v - base) / (1.f + expf(v)) : 1.f / (1.f + expf(-v));
    }
    if (renorm) {
        const float tot = wave_sum(w);
        w = tot > 0.f ? w / tot : 0.f;
    }
    if (lane < topk) {
        ids[t * topk + lane] = mine ? (int32_t)mine_id : -1;
        wts[t * topk + lane] = w;
    }
}

hipError_t launch_moe_route(const void* L, bool lf32, int64_t T, int E, int64_t ldl, int topk, int score, int renorm,
                            int32_t* ids, float* w, hipStream_t st) {
    const dim3 grid((unsigned)((T + kRouteWaves - 1) / kRouteWaves)), block(kRouteWaves * kWave);
#define TTQ_ROUTE(NV)                                                                                             \
    return lf32 ? launch_kernel(k_moe_route<NV, true>, grid, block, 0, st, nullptr, nullptr, L, T, E, ldl, topk,  \
                                score, renorm, ids, w)                                                            \
                : launch_kernel(k_moe_route<NV, false>, grid, block, 0, st, nullptr, nullptr, L, T, E, ldl, topk, \
                                score, renorm, ids, w)
    if (E <= 64) TTQ_ROUTE(1);
    if (E <= 128) TTQ_ROUTE(2);
    if (E <= 256) TTQ_ROUTE(4);
    if (E <= 512) TTQ_ROUTE(8);
    TTQ_ROUTE(16);
#undef TTQ_ROUTE
}

}  // namespace ttq
