// A gated mixture-of-experts layer on quantized experts, for few tokens:
//   Y[t] = sum_j w[t][j] Wd_e (h / s_down),  h = act(g) u,
//   [g; u] = Wgu_e (x_t / s_in),  e = ids[t][j],
// with every W = (code - zero) * step.  A slot (t, j) whose id names no
// expert adds nothing.
//
// Four launches.  The slots are grouped by expert (moe.hpp), so that an
// expert's codes are read once for all of its tokens (per tile of slots), and
// x / s is laid out as the products' operand; the first product's epilogue
// forms h with the slot's weight and 1 / s_down folded in and lays it out
// alike; the second leaves one fp32 row per slot (and slice of its channels),
// which are added here in slot order.  One or two tokens: moe_dot.hip; more, or
// other codes: moe_mfma.hip.
#include "common.hpp"
#include "launch.hpp"
#include "moe.hpp"

namespace ttq {

constexpr int kSumThreads = 64;

template <bool YF32>
__global__ __launch_bounds__(kSumThreads) void k_moe_sum(const float* __restrict__ P, int slices,
                                                         const int32_t* __restrict__ ids, int topk, int E, int64_t n,
                                                         int64_t M, void* __restrict__ Y, int64_t ldy) {
    const int64_t t = blockIdx.y, o = (int64_t)blockIdx.x * kSumThreads + threadIdx.x;
    if (o >= M) return;
    float y = 0.f;
    for (int j = 0; j < topk; ++j) {
        const int e = ids[t * topk + j];
        if (e < 0 || e >= E) continue;
        const float* p = P + (t * topk + j) * M + o;
        float v = 0.f;
        for (int s0 = 0; s0 < slices; s0 += 8) {  // eight loads together
            float x[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) x[u] = s0 + u < slices ? p[(s0 + u) * n * M] : 0.f;
#pragma unroll
            for (int u = 0; u < 8; ++u) v += x[u];
        }
        y += v;
    }
    if constexpr (YF32) ((float*)Y)[t * ldy + o] = y;
    else ((uint16_t*)Y)[t * ldy + o] = (uint16_t)f32_to_bf16(y);
}

hipError_t launch_moe_sum(const ttq_moe_args* a, const float* p, int slices, hipStream_t st) {
    const dim3 grid((unsigned)((a->M + kSumThreads - 1) / kSumThreads), (unsigned)a->T);
    const int64_t n = a->T * a->topk;
    return a->yt == TTQ_F32 ? launch_kernel(k_moe_sum<true>, grid, dim3(kSumThreads), 0, st, nullptr, nullptr, p, slices,
                                            a->ids, (int)a->topk, (int)a->E, n, a->M, a->Y, a->ldy)
                            : launch_kernel(k_moe_sum<false>, grid, dim3(kSumThreads), 0, st, nullptr, nullptr, p, slices,
                                            a->ids, (int)a->topk, (int)a->E, n, a->M, a->Y, a->ldy);
}

// Regions of both paths: an operand row takes at most 3 x 2 bytes per padded
// channel (the bf16 terms of fp32 X), digits less.
static MoeLayout layout(int64_t T, int64_t topk, int64_t K, int64_t I, int64_t M, int64_t E) {
    auto up = [](size_t n) { return (n + 255) / 256 * 256; };
    const int64_t n = T * topk, kp = moe_dot_pad(K), ip = moe_dot_pad(I);
    const int sl = moe_slices(n, E, I, M), sd = T == 1 || T == 2 ? moe_dot_slices(n, E, I, M, (int)T) : 1;
    MoeLayout L{};
    L.order = 0;
    L.tiles = L.order + up((size_t)n * 4);
    L.xt = L.tiles + up((size_t)moe_tiles(n, E, 1) * sizeof(MoeTile));
    L.xs = L.xt + up((size_t)n * kp * 6);
    L.h = L.xs + up((size_t)n * (kp / 16) * 4);
    L.hs = L.h + up((size_t)n * ip * 6);
    L.p = L.hs + up((size_t)n * (ip / 16) * 4);
    L.total = L.p + up((size_t)(sl > sd ? sl : sd) * n * M * 4);
    return L;
}

size_t moe_ws_bytes(int64_t T, int64_t topk, int64_t K, int64_t I, int64_t M, int64_t E) {
    return layout(T, topk, K, I, M, E).total;
}

hipError_t launch_moe(const ttq_moe_args* a, char* ws, hipStream_t st) {
    const MoeLayout L = layout(a->T, a->topk, a->K, a->I, a->M, a->E);
    return moe_dot_tile(a) > 0 ? launch_moe_dot(a, L, ws, st) : launch_moe_mfma(a, L, ws, st);
}

}  // namespace ttq
