// Shared by the kernels of the mixture-of-experts layer.
#pragma once

#include "common.hpp"
#include "launch.hpp"

namespace ttq {

struct MoeTile {
    int expert, first, count;   // `count` slots from position `first` of the slots sorted by expert
};

// Upper bound of the number of tiles of at most `tile` slots of one expert.
inline int64_t moe_tiles(int64_t n, int64_t E, int64_t tile) {
    const int64_t a = n < E ? n : E;
    return a + (n - a) / tile;
}

struct MoePlan {
    const int32_t* ids;
    int n, E, tile, ntiles;
    int32_t* order;
    MoeTile* tiles;
};

constexpr int kPlanThreads = 512;

// One workgroup of kPlanThreads: the slots grouped by expert into `order`
// and the tiles, unused ones with count 0.  The place of a slot within its
// expert depends on the timing of LDS atomics, and no result depends on it: a
// slot's products are those of its own row wherever that row stands.
__device__ __forceinline__ void moe_plan(const MoePlan& a) {
    __shared__ int cnt[kMoeMaxExperts], pos[kMoeMaxExperts];
    const int tid = threadIdx.x;
    for (int e = tid; e < a.E; e += kPlanThreads) cnt[e] = 0;
    __syncthreads();
    for (int i = tid; i < a.n; i += kPlanThreads) {
        const int e = a.ids[i];
        if (e >= 0 && e < a.E) atomicAdd(&cnt[e], 1);
    }
    __syncthreads();
    if (tid < kWave) {
        int p0 = 0, q0 = 0;                       // slots and tiles of the experts before this round's
        for (int b = 0; b < a.E; b += kWave) {
            const int e = b + tid;
            const int c = e < a.E ? cnt[e] : 0, nt = (c + a.tile - 1) / a.tile;
            int p = c, q = nt;
#pragma unroll
            for (int s = 1; s < kWave; s <<= 1) {
                const int pu = __shfl_up(p, s), qu = __shfl_up(q, s);
                if (tid >= s) {
                    p += pu;
                    q += qu;
                }
            }
            if (e < a.E) {
                const int first = p0 + p - c, tq = q0 + q - nt;
                pos[e] = first;
                for (int j = 0; j < nt; ++j)
                    a.tiles[tq + j] = MoeTile{e, first + j * a.tile, min(a.tile, c - j * a.tile)};
            }
            p0 += __shfl(p, kWave - 1);
            q0 += __shfl(q, kWave - 1);
        }
        for (int i = q0 + tid; i < a.ntiles; i += kWave) a.tiles[i] = MoeTile{0, 0, 0};
    }
    __syncthreads();
    for (int i = tid; i < a.n; i += kPlanThreads) {
        const int e = a.ids[i];
        if (e >= 0 && e < a.E) a.order[atomicAdd(&pos[e], 1)] = i;
    }
}

__device__ __forceinline__ float moe_act(float x, int act) {
    if (act == TTQ_ACT_SILU) return x / (1.f + expf(-x));
    const float u = 0.7978845608028654f * (x + 0.044715f * x * x * x);
    return x * (1.f - 1.f / (1.f + expf(2.f * u)));      // x (1 + tanh u) / 2
}

// Workspace regions (bytes from its start).
struct MoeLayout {
    size_t order, tiles, xt, xs, h, hs, p, total;
};

// y[t] = the sum over the token's slots that have an expert and over `slices`
// partial results of each, p [slices][T topk][M], in that order.
hipError_t launch_moe_sum(const ttq_moe_args* a, const float* p, int slices, hipStream_t st);

// ---- on the matrix cores (moe_mfma.hip): 4-bit codes, groups of 32 or more

constexpr int kMmTile = 16;                       // slots per tile

struct MoePrep {
    const void* X;
    int64_t ldx, K, kp, rows;
    const float* s;
    int64_t s_stride;
    const int32_t* ids;
    int topk, E;
    uint16_t* xt;               // [rows][terms][kp]
    float* xs;                  // [rows][kp / 16]: sums of 16 channels
};
struct MoeMm {
    const MoeTile* tiles;
    const int32_t* order;
    int64_t slots;
    const uint16_t* xt;         // operand rows: slot / div
    const float* xs;
    int64_t K, kp, rows;
    int div, per_slice, ksplit, act;
    const uint32_t* codes;
    const uint16_t* scale;
    const uint16_t* zero;
    const float* w;             // first product: h = act(g) u w / s_out
    const float* s_out;
    int64_t s_out_stride;
    uint16_t* ht;               // [slots][terms][hp]
    float* hs;
    int64_t hp;
    float* p;                   // second product: [slices][slots][rows]
};

bool moe_mfma_ok(const ttq_moe_args* a);
int64_t moe_pad(int64_t K);
int moe_slices(int64_t n, int64_t E, int64_t I, int64_t M);
hipError_t launch_moe_mfma(const ttq_moe_args* a, const MoeLayout& L, char* ws, hipStream_t st);

}  // namespace ttq
