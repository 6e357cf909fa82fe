// Shared by the kernels of the mixture-of-experts layer.
#pragma once

#include "common.hpp"
#include "launch.hpp"
#include "lds_dma.hpp"

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
constexpr int kSimds = 4 * 256;                   // of the chip

// One workgroup of kPlanThreads: the slots grouped by expert (without ids: all
// of expert 0, in their order) into `order`
// and the tiles, unused ones with count 0.  The place of a slot within its
// expert depends on the timing of LDS atomics, and no result depends on it: a
// slot's products are those of its own row wherever that row stands.
__device__ __forceinline__ void moe_plan(const MoePlan& a) {
    __shared__ int cnt[kMoeMaxExperts], pos[kMoeMaxExperts];
    const int tid = threadIdx.x;
    if (a.ids == nullptr) {
        for (int i = tid; i < a.n; i += kPlanThreads) a.order[i] = i;
        for (int j = tid; j < a.ntiles; j += kPlanThreads)
            a.tiles[j] = MoeTile{0, j * a.tile, min(a.tile, a.n - j * a.tile)};
        return;
    }
    for (int e = tid; e < a.E; e += kPlanThreads) cnt[e] = 0;
    __syncthreads();
    for (int i = tid; i < a.n; i += kPlanThreads) {
        const int e = a.ids[i];
        if (e >= 0 && e < a.E) atomicAdd(&cnt[e], 1);
    }
    __syncthreads();
    if (tid < kWave) {
        int p0 = 0, q0 = 0;                       // slots and tiles of the experts before these 64
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
    // x (1 + tanh u) / 2 without a difference of near numbers (1 + tanh u has
    // no correct digit left below x = -5).
    const float u = 0.7978845608028654f * (x + 0.044715f * x * x * x);
    return x / (1.f + expf(-2.f * u));
}

// Workspace regions (bytes from its start).
struct MoeLayout {
    size_t order, tiles, xt, xs, h, hs, p, total;
};

// y[t] = the sum over the token's slots that have an expert and over `slices`
// partial results of each, p [slices][T topk][M], in that order.
hipError_t launch_moe_sum(const ttq_moe_args* a, const float* p, int slices, hipStream_t st);

// ---- on the matrix cores (moe_mfma.hip)

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
    int div, group, per_slice, ksplit, act, xbytes;
    const uint32_t* codes;
    const uint16_t* scale;
    const uint16_t* zero;
    const float* w;             // first product: h = act(g) u w / s_out
    const float* s_out;
    int64_t s_out_stride;
    uint16_t* ht;               // [slots][terms][hp]
    float* hs;
    int64_t hp;
    float* p;                   // second product: [slices][slots][ldp], from its row's place
    int64_t ldp;
};

// Eight channels from k0 of token t, divided by the scales of expert e.
template <bool XF32>
__device__ __forceinline__ void moe_load_scaled(float (&x)[8], const MoePrep& a, int64_t t, int64_t e, int64_t k0) {
    if constexpr (XF32) {
        const f32x4 u = *(const f32x4*)((const float*)a.X + t * a.ldx + k0);
        const f32x4 v = *(const f32x4*)((const float*)a.X + t * a.ldx + k0 + 4);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            x[j] = u[j];
            x[4 + j] = v[j];
        }
    } else {
        const u32x4 u = *(const u32x4*)((const uint16_t*)a.X + t * a.ldx + k0);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            x[2 * j] = bf16lo_to_f32(u[j]);
            x[2 * j + 1] = bf16hi_to_f32(u[j]);
        }
    }
    const float* s = a.s + e * a.s_stride + k0;
    const f32x4 u = *(const f32x4*)s, v = *(const f32x4*)(s + 4);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        x[j] /= u[j];
        x[4 + j] /= v[j];
    }
}

// Descriptor of `bytes` bytes of fp16 values from p, its base aligned down to
// a word; `adj` (0 or 2) goes onto the offsets.
__device__ __forceinline__ rsrc_t moe_half_rsrc(const uint16_t* p, int64_t bytes, uint32_t& adj) {
    adj = (uint32_t)((uintptr_t)p & 2);
    return make_rsrc((const char*)p - adj, (bytes + adj + 3) & ~(int64_t)3);
}
// NH fp16 values (4, 8 or 16) at byte offset `off` as packed words, in loads
// of up to 16 bytes; W2: the offset may lie within a word (rows of an odd
// number of groups), one word more is loaded and all are shifted.
template <int NH, bool W2>
__device__ __forceinline__ void moe_load_halves(uint32_t (&d)[NH / 2], rsrc_t r, uint32_t off) {
    const uint32_t at = W2 ? off & ~2u : off;
    uint32_t w[NH / 2 + 1];
    w[NH / 2] = 0;
    if constexpr (NH >= 8) {
#pragma unroll
        for (int h = 0; h < NH / 8; ++h) {
            const u32x4 a = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, (int)(at + 16 * h), 0, 0));
#pragma unroll
            for (int v = 0; v < 4; ++v) w[4 * h + v] = a[v];
        }
    } else {
        const u32x2 a = __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(r, (int)at, 0, 0));
        w[0] = a[0];
        w[1] = a[1];
    }
    if constexpr (W2) w[NH / 2] = __builtin_amdgcn_raw_buffer_load_b32(r, (int)(at + 2 * NH), 0, 0);
#pragma unroll
    for (int v = 0; v < NH / 2; ++v) d[v] = W2 ? __builtin_amdgcn_alignbit(w[v + 1], w[v], (off & 2) * 8) : w[v];
}
// One of a word's two fp16 values.
__device__ __forceinline__ float half_at(uint32_t d, bool hi) { return f16_to_f32((uint16_t)(hi ? d >> 16 : d & 0xFFFFu)); }
// Whether the rows of steps and zeros need W2.
inline bool moe_w2(const uint16_t* scale, const uint16_t* zero, int64_t groups) {
    return groups % 2 != 0 || (uintptr_t)scale % 4 != 0 || (uintptr_t)zero % 4 != 0;
}

// The rows of X as the first product's operand, kp padded channels.
inline MoePrep moe_prep_of(const ttq_moe_args* a, int64_t kp) {
    MoePrep pr{};
    pr.X = a->X; pr.ldx = a->ldx; pr.K = a->K; pr.kp = kp;
    pr.s = a->gate_up.s; pr.s_stride = a->gate_up.s_stride;
    pr.rows = pr.s_stride ? a->T * a->topk : a->T; pr.ids = a->ids; pr.topk = (int)a->topk; pr.E = (int)a->E;
    return pr;
}

int64_t moe_pad(int64_t K);
int moe_slices(int64_t n, int64_t E, int64_t I, int64_t M);
hipError_t launch_moe_mfma(const ttq_moe_args* a, const MoeLayout& L, char* ws, hipStream_t st);

// ---- integer dot products (moe_dot.hip): 4-bit codes, groups of 32 or more,
// one or two tokens

struct MoeDot {
    const MoeTile* tiles;
    const int32_t* order;
    int64_t slots;
    const uint32_t* xq;         // operand rows: slot / div
    int64_t K, kp, rows;
    int div, per_slice, ksplit, act;
    const uint32_t* codes;
    const uint16_t* scale;
    const uint16_t* zero;
    const float* w;             // first product: h = act(g) u w / s_out
    const float* s_out;
    int64_t s_out_stride;
    uint32_t* hq;               // [slots]
    int64_t hp;
    float* p;                   // second product: [slices][slots][rows]
};

int moe_dot_tile(const ttq_moe_args* a);          // slots per tile; 0: not this path
int64_t moe_dot_pad(int64_t K);
int moe_dot_slices(int64_t n, int64_t E, int64_t I, int64_t M, int tile);
hipError_t launch_moe_dot(const ttq_moe_args* a, const MoeLayout& L, char* ws, hipStream_t st);

}  // namespace ttq
