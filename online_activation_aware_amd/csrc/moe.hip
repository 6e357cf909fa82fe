// A gated mixture-of-experts layer on quantized experts, for few tokens:
//   Y[t] = sum_j w[t][j] Wd_e (h / s_down),  h = act(g) u,
//   [g; u] = Wgu_e (x_t / s_in),  e = ids[t][j],
// with every W = (code - zero) * step.  A slot (t, j) whose id names no
// expert adds nothing.
//
// The slots are grouped by expert once (k_moe_plan), so that an expert's
// codes are read once for all of its tokens (per tile of slots); the products
// apply the group's step and zero to sums, step (sum q x - zero sum x), in
// fp32.  h is kept in fp32, multiplied by w / s_down: the second product then
// needs neither.  Its results, one row per slot, are added in slot order.
#include "codes.hpp"
#include "common.hpp"
#include "launch.hpp"
#include "moe.hpp"

namespace ttq {

__global__ __launch_bounds__(kPlanThreads) void k_moe_plan(MoePlan a) { moe_plan(a); }

// ------------------------------------------------------------------ products

// One of the layer's two products, for tiles of slots of one expert.
struct MoeProduct {
    const MoeTile* tiles;
    const int32_t* order;       // slots sorted by expert
    const void* X;              // rows of K: tokens (row slot / topk), or h (row slot)
    int64_t ldx, K, rows;       // rows: outputs per slot
    int topk, group, act;
    const float* s;             // per expert, at s_stride
    int64_t s_stride;
    const uint32_t* codes;
    const uint16_t* scale;
    const uint16_t* zero;
    const float* w;             // weight of each slot
    const float* s_out;         // scales of the second product's input
    int64_t s_out_stride;
    float* out;                 // [slots][rows]
};

constexpr int kMtRows = 16;                       // code rows per workgroup
constexpr int kMtTok = 4;                         // slots per tile
constexpr int kMtWaves = 8;
constexpr int kMtPiece = kTChan * kWave;          // channels a wave covers at once

// SG: groups per 32-channel field (2 for groups of 16).  GU: the first
// product, rows i and I + i for 8 consecutive i; else the second, 16 rows.
template <int BITS, int SG, bool XF32, bool GU>
__global__ __launch_bounds__(kMtWaves * kWave) void k_moe_rows(MoeProduct a) {
    constexpr int SGC = kTChan / SG;
    constexpr int NV = kMtRows * kMtTok;
    __shared__ float red[kMtWaves][NV];
    const MoeTile tl = a.tiles[blockIdx.y];
    if (tl.count == 0) return;
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int ns = blockDim.x / kWave;
    const int64_t K = a.K, wpr = K * BITS / 32, gpr = K / a.group;
    const int64_t R = GU ? 2 * a.rows : a.rows;   // code rows of an expert
    const uint32_t* codes = a.codes + (int64_t)tl.expert * R * wpr;
    const uint16_t* scale = a.scale + (int64_t)tl.expert * R * gpr;
    const uint16_t* zero = a.zero + (int64_t)tl.expert * R * gpr;
    const int64_t o0 = (int64_t)blockIdx.x * (GU ? kMtRows / 2 : kMtRows);
    int slot[kMtTok];
#pragma unroll
    for (int t = 0; t < kMtTok; ++t) slot[t] = a.order[tl.first + min(t, tl.count - 1)];

    float acc[kMtRows][kMtTok];
#pragma unroll
    for (int r = 0; r < kMtRows; ++r)
#pragma unroll
        for (int t = 0; t < kMtTok; ++t) acc[r][t] = 0.f;

    for (int64_t p = wave; p * kMtPiece < K; p += ns) {
        const int64_t k0 = p * kMtPiece + (int64_t)lane * kTChan;
        if (k0 >= K) continue;                    // K % 32 == 0: a field is all in or all out
        float xs[kMtTok][kTChan], S[kMtTok][SG];
#pragma unroll
        for (int t = 0; t < kMtTok; ++t) {
            const int64_t row = GU ? slot[t] / a.topk : slot[t];
#pragma unroll
            for (int v = 0; v < kTChan / 4; ++v) {
                float x[4];
                if constexpr (XF32) {
                    const f32x4 f = *(const f32x4*)((const float*)a.X + row * a.ldx + k0 + 4 * v);
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[e] = f[e];
                } else {
                    const u32x2 f = *(const u32x2*)((const uint16_t*)a.X + row * a.ldx + k0 + 4 * v);
                    x[0] = bf16lo_to_f32(f[0]); x[1] = bf16hi_to_f32(f[0]);
                    x[2] = bf16lo_to_f32(f[1]); x[3] = bf16hi_to_f32(f[1]);
                }
                if constexpr (GU) {
                    const f32x4 s = *(const f32x4*)(a.s + tl.expert * a.s_stride + k0 + 4 * v);
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[e] *= __builtin_amdgcn_rcpf(s[e]);
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) xs[t][4 * v + e] = x[e];
            }
#pragma unroll
            for (int h = 0; h < SG; ++h) {
                float sum = xs[t][h * SGC];
#pragma unroll
                for (int i = 1; i < SGC; ++i) sum += xs[t][h * SGC + i];
                S[t][h] = sum;
            }
        }
#pragma unroll
        for (int r = 0; r < kMtRows; ++r) {
            int64_t o;
            if constexpr (GU) o = min(o0 + (r & 7), a.rows - 1) + (r >= 8 ? a.rows : 0);
            else o = min(o0 + r, a.rows - 1);
            CodeWords<BITS> cw;
            load_codes<BITS>(cw, codes + o * wpr + k0 * BITS / 32);
            float q[kTChan];
            field_codes<BITS>(cw, q);
#pragma unroll
            for (int h = 0; h < SG; ++h) {
                const int64_t g = o * gpr + (SG == 2 ? k0 / 16 + h : k0 / a.group);
                const float df = f16_to_f32(scale[g]), zf = f16_to_f32(zero[g]);
#pragma unroll
                for (int t = 0; t < kMtTok; ++t) {
                    if (t >= tl.count) continue;  // uniform
                    float d = q[h * SGC] * xs[t][h * SGC];
#pragma unroll
                    for (int i = 1; i < SGC; ++i) d = __builtin_fmaf(q[h * SGC + i], xs[t][h * SGC + i], d);
                    acc[r][t] = __builtin_fmaf(df, __builtin_fmaf(-zf, S[t][h], d), acc[r][t]);
                }
            }
            __builtin_amdgcn_sched_barrier(0);    // rows are not interleaved (registers)
        }
    }

    // Sum over the wave (lane l ends with value l), then over the waves.
    float v[NV];
#pragma unroll
    for (int r = 0; r < kMtRows; ++r)
#pragma unroll
        for (int t = 0; t < kMtTok; ++t) v[r * kMtTok + t] = acc[r][t];
    int idx = 0;
#pragma unroll
    for (int m = 32, n = NV; m >= 1; m >>= 1) {
        const int half = n / 2;
        const bool up = (lane & m) != 0;
        const uint32_t um = up ? 0xFFFFFFFFu : 0u;
#pragma unroll
        for (int i = 0; i < half; ++i) {
            // Selects on the bit patterns: no dynamic array index.
            const uint32_t x = __builtin_bit_cast(uint32_t, v[i]), y = __builtin_bit_cast(uint32_t, v[i + half]);
            const float send = __builtin_bit_cast(float, (x & um) | (y & ~um));
            const float keep = __builtin_bit_cast(float, (y & um) | (x & ~um));
            v[i] = keep + __shfl_xor(send, m);
        }
        idx = 2 * idx + (up ? 1 : 0);
        n = half;
    }
    red[wave][idx] = v[0];
    __syncthreads();
    if (threadIdx.x >= NV) return;                // the first wave
    const int vi = threadIdx.x, r = vi / kMtTok, t = vi % kMtTok;
    float sum = red[0][vi];
    for (int w = 1; w < ns; ++w) sum += red[w][vi];
    int myslot = slot[0];
#pragma unroll
    for (int u = 1; u < kMtTok; ++u) myslot = t == u ? slot[u] : myslot;
    if constexpr (GU) {
        const float up = __shfl(sum, (vi + 8 * kMtTok) & (kWave - 1));
        const int64_t o = o0 + r;
        if (r < 8 && o < a.rows && t < tl.count) {
            const float f = a.w[myslot] / a.s_out[tl.expert * a.s_out_stride + o];
            a.out[(int64_t)myslot * a.rows + o] = moe_act(sum, a.act) * up * f;
        }
    } else {
        const int64_t o = o0 + r;
        if (o < a.rows && t < tl.count) a.out[(int64_t)myslot * a.rows + o] = sum;
    }
}

constexpr int kSumThreads = 64;

template <bool YF32>
__global__ __launch_bounds__(kSumThreads) void k_moe_sum(const float* __restrict__ P, int slices, const int32_t* __restrict__ ids,
                                                 int topk, int E, int64_t n, int64_t M, void* __restrict__ Y,
                                                 int64_t ldy) {
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

// ------------------------------------------------------------------ host

// Regions of all paths: an operand row takes at most 3 x 2 bytes per padded
// channel (the bf16 terms of fp32 X), digits and fp32 h less.
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

template <bool XF32, bool GU>
static hipError_t launch_rows(const MoeProduct& p, int bits, int64_t ntiles, hipStream_t st) {
    const int64_t np = (p.K + kMtPiece - 1) / kMtPiece;
    const int64_t rounds = (np + kMtWaves - 1) / kMtWaves;
    const int ns = (int)((np + rounds - 1) / rounds);
    const int per = GU ? kMtRows / 2 : kMtRows;
    const dim3 grid((unsigned)((p.rows + per - 1) / per), (unsigned)ntiles), block(ns * kWave);
#define TTQ_ROWS(B)                                                                                          \
    return p.group == 16 ? launch_kernel(k_moe_rows<B, 2, XF32, GU>, grid, block, 0, st, nullptr, nullptr, p) \
                         : launch_kernel(k_moe_rows<B, 1, XF32, GU>, grid, block, 0, st, nullptr, nullptr, p)
    switch (bits) {
        case 2: TTQ_ROWS(2);
        case 3: TTQ_ROWS(3);
        case 4: TTQ_ROWS(4);
        case 5: TTQ_ROWS(5);
    }
#undef TTQ_ROWS
    return hipErrorInvalidValue;
}

hipError_t launch_moe(const ttq_moe_args* a, char* ws, hipStream_t st) {
    const int64_t n = a->T * a->topk;
    const MoeLayout L = layout(a->T, a->topk, a->K, a->I, a->M, a->E);
    if (moe_dot_tile(a) > 0) return launch_moe_dot(a, L, ws, st);
    if (moe_mfma_ok(a)) return launch_moe_mfma(a, L, ws, st);
    int32_t* order = (int32_t*)(ws + L.order);
    MoeTile* tiles = (MoeTile*)(ws + L.tiles);
    const int64_t nt = moe_tiles(n, a->E, kMtTok);
    const MoePlan pl{a->ids, (int)n, (int)a->E, kMtTok, (int)nt, order, tiles};
    if (hipError_t e = launch_kernel(k_moe_plan, dim3(1), dim3(kPlanThreads), 0, st, nullptr, nullptr, pl)) return e;
    MoeProduct p{};
    p.tiles = tiles; p.order = order;
    p.X = a->X; p.ldx = a->ldx; p.K = a->K; p.rows = a->I; p.topk = (int)a->topk; p.group = a->group; p.act = a->act;
    p.s = a->gate_up.s; p.s_stride = a->gate_up.s_stride;
    p.codes = (const uint32_t*)a->gate_up.codes; p.scale = a->gate_up.scale_f16; p.zero = a->gate_up.zero_f16;
    p.w = a->w; p.s_out = a->down.s; p.s_out_stride = a->down.s_stride;
    p.out = (float*)(ws + L.h);
    if (hipError_t e = a->xt == TTQ_F32 ? launch_rows<true, true>(p, a->bits, nt, st)
                                        : launch_rows<false, true>(p, a->bits, nt, st))
        return e;
    MoeProduct d{};
    d.tiles = tiles; d.order = order;
    d.X = ws + L.h; d.ldx = a->I; d.K = a->I; d.rows = a->M; d.topk = 1; d.group = a->group;
    d.codes = (const uint32_t*)a->down.codes; d.scale = a->down.scale_f16; d.zero = a->down.zero_f16;
    d.out = (float*)(ws + L.p);
    if (hipError_t e = launch_rows<true, false>(d, a->bits, nt, st)) return e;
    return launch_moe_sum(a, d.out, 1, st);
}

}  // namespace ttq
