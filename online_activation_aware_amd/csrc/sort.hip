// Tokens sorted by expert, their rows copied in that order, and the way back.
//
// Sort: slots (token, j) by the expert ids[t][j], stably, so that every result
// is the same each time; a slot whose id names no expert has no row.
//   offsets[e]: rows of the experts before e;  order[r]: row r's slot;
//   pos[slot]: its row.
// A workgroup owns consecutive slots and each of its 16 waves a run of them.
// Per 64 slots the lanes of equal experts are found by a ballot per bit of the
// id, so that a wave counts without atomics: the first such lane adds their
// number.  Counts of waves (in LDS) and of workgroups (in memory, by a launch
// of its own where there are several) become the places where their slots of
// each expert begin.  Bound by latency: 49152 slots of 160 experts two launches of
// 5 us, 32 slots one of 4.
//
// Rows are copied (gather), added (combine) and differentiated (combine_grad)
// by token, through pos: a token's row is read or written once for all of its
// slots, in whole vectors of 16 bytes.  Bound by memory: 8192 tokens of 2048 bf16
// values, 6 slots each, gathered (a quarter of the slots without an expert) 35 us,
// combined 44 (5.3 TB/s); the gradient for 4096 tokens of 4096 values, 2 slots
// each, 36 (4.7 TB/s).
#include <algorithm>

#include "common.hpp"
#include "launch.hpp"
#include "lds_dma.hpp"
#include "sort.hpp"
#include "wave.hpp"

namespace ttq {

size_t moe_sort_ws_bytes(int64_t n, int64_t E) {
    return sort_blocks(n) > 1 ? (size_t)(sort_blocks(n) * E) * 4 : 0;
}

template <bool PLACE>
__global__ __launch_bounds__(kSortThreads) void k_moe_sort(SortArgs a) {
    sort_block<PLACE>(a, blockIdx.x, gridDim.x);
}

hipError_t launch_moe_sort(const int32_t* ids, int64_t n, int E, int32_t* offsets, int32_t* order, int32_t* pos,
                           int32_t* ws, hipStream_t st) {
    const SortArgs a = sort_args(ids, n, E, offsets, order, pos, ws);
    const dim3 grid((unsigned)sort_blocks(n)), block(kSortThreads);
    if (grid.x > 1) {
        const hipError_t e = launch_kernel(k_moe_sort<false>, grid, block, 0, st, nullptr, nullptr, a);
        if (e != hipSuccess) return e;
    }
    return launch_kernel(k_moe_sort<true>, grid, block, 0, st, nullptr, nullptr, a);
}

// ------------------------------------------------------------------ rows

// 256 lanes take the pieces (16 bytes of the sorted rows) of one token or of
// several, whole waves of one token, so that pos and w are scalars.  (A division
// for each piece's token costs more than the copy.)
constexpr int kMoveThreads = 256;

struct Moves {
    int tokens, lanes;                            // of a workgroup; of a token
    dim3 grid;
};
static Moves moves(int64_t T, int64_t pieces) {
    int lanes = kWave;
    while (lanes < kMoveThreads && lanes < pieces) lanes *= 2;
    const int tokens = kMoveThreads / lanes;
    return {tokens, lanes,
            dim3((unsigned)std::min<int64_t>((T + tokens - 1) / tokens, 1 << 20),
                 (unsigned)std::min<int64_t>((pieces + lanes - 1) / lanes, 1024))};
}

// One row piece of 16 bytes, or its `n` elements of ES bytes at the row's end.
template <int ES>
__device__ __forceinline__ u32x4 load_piece(const char* p, int n) {
    u32x4 v = {0, 0, 0, 0};
    if (n >= 16 / ES) return *(const u32x4*)p;
    if constexpr (ES == 4) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < n) v[i] = ((const uint32_t*)p)[i];
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) v[i / 2] |= (uint32_t)((const uint16_t*)p)[i] << (16 * (i & 1));
    }
    return v;
}
template <int ES>
__device__ __forceinline__ void store_piece(char* p, int n, const u32x4& v) {
    if (n >= 16 / ES) {
        *(u32x4*)p = v;
    } else if constexpr (ES == 4) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < n) ((uint32_t*)p)[i] = v[i];
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) ((uint16_t*)p)[i] = (uint16_t)(v[i / 2] >> (16 * (i & 1)));
    }
}

// The token of this wave in turn i of its workgroup's, and its lane among the
// token's.
__device__ __forceinline__ int64_t move_token(int64_t i, int tokens, int lanes) {
    return i * tokens + __builtin_amdgcn_readfirstlane((int)threadIdx.x / lanes);
}

template <int ES>
__global__ __launch_bounds__(kMoveThreads) void k_moe_gather(const char* __restrict__ X, int64_t T, int64_t K,
                                                             int64_t ldx, const int32_t* __restrict__ pos, int topk,
                                                             char* __restrict__ R, int64_t rows, int64_t ldr,
                                                             int tokens, int lanes) {
    constexpr int V = 16 / ES;
    const int64_t step = (int64_t)V * lanes * gridDim.y;
    for (int64_t i = blockIdx.x; i * tokens < T; i += gridDim.x) {
        const int64_t t = move_token(i, tokens, lanes);
        if (t >= T) break;
        for (int64_t k = (int64_t)V * (blockIdx.y * lanes + threadIdx.x % lanes); k < K; k += step) {
            const int n = (int)min(K - k, (int64_t)V);
            const u32x4 v = load_piece<ES>(X + (t * ldx + k) * ES, n);
            for (int j = 0; j < topk; ++j) {
                const int64_t r = pos[t * topk + j];
                if (r >= 0 && r < rows) store_piece<ES>(R + (r * ldr + k) * ES, n, v);
            }
        }
    }
}

hipError_t launch_moe_gather(const void* X, int es, int64_t T, int64_t K, int64_t ldx, const int32_t* pos, int topk,
                             void* R, int64_t rows, int64_t ldr, hipStream_t st) {
    const Moves m = moves(T, (K * es + 15) / 16);
    return es == 4 ? launch_kernel(k_moe_gather<4>, m.grid, dim3(kMoveThreads), 0, st, nullptr, nullptr, (const char*)X, T,
                                   K, ldx, pos, topk, (char*)R, rows, ldr, m.tokens, m.lanes)
                   : launch_kernel(k_moe_gather<2>, m.grid, dim3(kMoveThreads), 0, st, nullptr, nullptr, (const char*)X, T,
                                   K, ldx, pos, topk, (char*)R, rows, ldr, m.tokens, m.lanes);
}

// A piece's values in fp32.
template <bool F32>
struct Piece {
    static constexpr int V = F32 ? 4 : 8;
    u32x4 w;
    __device__ __forceinline__ void load(const void* p, int64_t at, int n) {
        w = load_piece<F32 ? 4 : 2>((const char*)p + at * (F32 ? 4 : 2), n);
    }
    __device__ __forceinline__ float operator[](int i) const {
        const uint32_t u = w[F32 ? i : i / 2];    // (a copy: a bit cast of the element takes the first)
        if constexpr (F32) return __builtin_bit_cast(float, u);
        return i % 2 ? bf16hi_to_f32(u) : bf16lo_to_f32(u);
    }
};

// A token's V values from index k on.
template <bool YF32, int V>
__device__ __forceinline__ void store_values(void* Y, int64_t at, int n, int yvec, const float (&y)[V]) {
    if (!YF32 && V == 8 && yvec && n >= 8) {
        *(u32x4*)((uint16_t*)Y + at) = u32x4{pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]), pack_bf16x2(y[4 % V], y[5 % V]),
                                             pack_bf16x2(y[6 % V], y[7 % V])};
        return;
    }
#pragma unroll
    for (int q = 0; q < V; q += 4)
        if (q < n) store_y4<YF32>(Y, at + q, n - q, yvec, f32x4{y[q], y[q + 1], y[q + 2], y[q + 3]});
}

constexpr int kCombineSlots = 4;                  // rows requested together

template <bool RF32, bool YF32>
__global__ __launch_bounds__(kMoveThreads) void k_moe_combine(const void* __restrict__ R, int64_t rows, int64_t ldr,
                                                              const int32_t* __restrict__ pos,
                                                              const float* __restrict__ w, int64_t T, int topk,
                                                              int64_t M, void* __restrict__ Y, int64_t ldy, int yvec,
                                                              int tokens, int lanes) {
    constexpr int V = Piece<RF32>::V;
    const int64_t step = (int64_t)V * lanes * gridDim.y;
    for (int64_t i = blockIdx.x; i * tokens < T; i += gridDim.x) {
        const int64_t t = move_token(i, tokens, lanes);
        if (t >= T) break;
        for (int64_t k = (int64_t)V * (blockIdx.y * lanes + threadIdx.x % lanes); k < M; k += step) {
            const int n = (int)min(M - k, (int64_t)V);
            float y[V] = {};
            for (int j0 = 0; j0 < topk; j0 += kCombineSlots) {
                Piece<RF32> v[kCombineSlots];
                bool have[kCombineSlots];
                float f[kCombineSlots];
#pragma unroll
                for (int u = 0; u < kCombineSlots; ++u) {
                    const int64_t r = j0 + u < topk ? pos[t * topk + j0 + u] : -1;
                    have[u] = r >= 0 && r < rows;
                    f[u] = 1.f;
                    if (have[u]) {
                        v[u].load(R, r * ldr + k, n);
                        if (w) f[u] = w[t * topk + j0 + u];
                    }
                }
#pragma unroll
                for (int u = 0; u < kCombineSlots; ++u)
                    if (have[u])
#pragma unroll
                        for (int c = 0; c < V; ++c) y[c] = __builtin_fmaf(f[u], v[u][c], y[c]);
            }
            store_values<YF32, V>(Y, t * ldy + k, n, yvec, y);
        }
    }
}

hipError_t launch_moe_combine(const void* R, bool rf32, int64_t rows, int64_t ldr, const int32_t* pos, const float* w,
                              int64_t T, int topk, int64_t M, void* Y, bool yf32, int64_t ldy, hipStream_t st) {
    const Moves m = moves(T, rf32 ? (M + 3) / 4 : (M + 7) / 8);
    const int yvec = (uintptr_t)Y % 16 == 0 && ldy * (yf32 ? 4 : 2) % 16 == 0;
#define TTQ_COMBINE(RF, YF)                                                                                              \
    return launch_kernel(k_moe_combine<RF, YF>, m.grid, dim3(kMoveThreads), 0, st, nullptr, nullptr, R, rows, ldr, pos, w, T, \
                         topk, M, Y, ldy, yvec, m.tokens, m.lanes)
    if (rf32) {
        if (yf32) TTQ_COMBINE(true, true);
        TTQ_COMBINE(true, false);
    }
    if (yf32) TTQ_COMBINE(false, true);
    TTQ_COMBINE(false, false);
#undef TTQ_COMBINE
}

// A workgroup a token: for each slot dR's row and dw.  The token's row of dY is
// held in registers where it has at most kHeld pieces a lane, else read again for
// each slot (from the cache).  dw: a lane's products in the order of their
// columns, then the wave's and the waves' sums in a fixed order, in fp32.
constexpr int kHeld = 2;

template <bool YF32, bool RF32>
__global__ __launch_bounds__(kMoveThreads) void k_moe_combine_grad(const void* __restrict__ dY, int64_t lddy,
                                                                   const void* __restrict__ R, int64_t rows,
                                                                   int64_t ldr, const int32_t* __restrict__ pos,
                                                                   const float* __restrict__ w, int64_t T, int topk,
                                                                   int64_t M, void* __restrict__ dR, int64_t lddr,
                                                                   float* __restrict__ dw) {
    constexpr int V = Piece<RF32>::V, Q = V / Piece<YF32>::V > 0 ? V / Piece<YF32>::V : 1;
    __shared__ float part[kRouteMaxTopk][kMoveThreads / kWave];
    const int lane = threadIdx.x & (kWave - 1), wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    auto row = [&](int64_t t, int64_t k, int n, float (&g)[V]) __attribute__((always_inline)) {
        if constexpr (YF32 == RF32 || YF32) {     // one vector of dY, or two of fp32
#pragma unroll
            for (int q = 0; q < Q; ++q) {
                Piece<YF32> p;
                p.load(dY, t * lddy + k + q * Piece<YF32>::V, max(n - q * Piece<YF32>::V, 0));
#pragma unroll
                for (int c = 0; c < Piece<YF32>::V; ++c) g[q * Piece<YF32>::V + c] = p[c];
            }
        } else {                                  // half a vector of bf16
#pragma unroll
            for (int c = 0; c < V; ++c) g[c] = c < n ? bf16_to_f32(((const uint16_t*)dY)[t * lddy + k + c]) : 0.f;
        }
    };
    const int64_t step = (int64_t)V * kMoveThreads, first = (int64_t)V * threadIdx.x;
    const bool held = M <= kHeld * step;
    for (int64_t t = blockIdx.x; t < T; t += gridDim.x) {
        float g[kHeld][V];
        if (held)
#pragma unroll
            for (int u = 0; u < kHeld; ++u) {
                const int64_t k = first + u * step;
                if (k < M) row(t, k, (int)min(M - k, (int64_t)V), g[u]);
            }
        for (int j = 0; j < topk; ++j) {
            const int64_t r = pos[t * topk + j];
            const bool have = r >= 0 && r < rows;
            float dot = 0.f;
            if (have) {
                const float f = w ? w[t * topk + j] : 1.f;
                auto piece = [&](int64_t k, const float (&gy)[V]) __attribute__((always_inline)) {
                    const int n = (int)min(M - k, (int64_t)V);
                    if (dw) {
                        Piece<RF32> v;
                        v.load(R, r * ldr + k, n);    // (zeros behind the row's end)
#pragma unroll
                        for (int c = 0; c < V; ++c)
                            if (c < n) dot = __builtin_fmaf(gy[c], v[c], dot);
                    }
                    if (dR) {
                        float d[V];
#pragma unroll
                        for (int c = 0; c < V; ++c) d[c] = f * gy[c];
                        store_values<RF32, V>(dR, r * lddr + k, n, 1, d);
                    }
                };
                if (held) {
#pragma unroll
                    for (int u = 0; u < kHeld; ++u)
                        if (first + u * step < M) piece(first + u * step, g[u]);
                } else {
                    for (int64_t k = first; k < M; k += step) {
                        row(t, k, (int)min(M - k, (int64_t)V), g[0]);
                        piece(k, g[0]);
                    }
                }
            }
            if (dw) {
                dot = wave_sum(dot);
                if (lane == 0) part[j][wave] = have ? dot : 0.f;
            }
        }
        if (dw) {
            __syncthreads();
            if ((int)threadIdx.x < topk) {
                float s = 0.f;
#pragma unroll
                for (int v = 0; v < kMoveThreads / kWave; ++v) s += part[threadIdx.x][v];
                dw[t * topk + threadIdx.x] = s;
            }
            __syncthreads();
        }
    }
}

hipError_t launch_moe_combine_grad(const void* dY, bool yf32, int64_t lddy, const void* R, bool rf32, int64_t rows,
                                   int64_t ldr, const int32_t* pos, const float* w, int64_t T, int topk, int64_t M,
                                   void* dR, int64_t lddr, float* dw, hipStream_t st) {
    const dim3 grid((unsigned)std::min<int64_t>(T, 1 << 20)), block(kMoveThreads);
#define TTQ_GRAD(YF, RF)                                                                                             \
    return launch_kernel(k_moe_combine_grad<YF, RF>, grid, block, 0, st, nullptr, nullptr, dY, lddy, R, rows, ldr, pos, w, T, \
                         topk, M, dR, lddr, dw)
    if (yf32) {
        if (rf32) TTQ_GRAD(true, true);
        TTQ_GRAD(true, false);
    }
    if (rf32) TTQ_GRAD(false, true);
    TTQ_GRAD(false, false);
#undef TTQ_GRAD
}

}  // namespace ttq
