// Products of 8-bit codes with scales for each row of either side:
//   Y[t][o] = x_scale[t] w_scale[o] sum_j X[t][j] W[o][j],
// the sum exact in int32 on the matrix cores (K <= 2^17), for one matrix or for
// rows sorted by expert that multiply their own expert's; optionally
//   Y[t][o] = act(g) u / s[o],  g and u the products with rows o and M + o of W.
#include <algorithm>

#include "i8.hpp"

namespace ttq {

constexpr int kStreamRows = 16;                   // rows of W a workgroup

// W streamed once per tile of 16 NT rows of X: a workgroup owns 16 rows of W (16
// of gate and of up), its waves share out the channels, 64 at a time, and add
// their sums through LDS.
template <int NT, bool GATE, bool YF32>
__global__ __launch_bounds__(NT <= 2 ? 1024 : 512) void k_i8_stream(I8Product p) {
    constexpr int NW = NT <= 2 ? 16 : 8, G = GATE ? 2 : 1;
    __shared__ i32x4 sums[NW][G][NT][kWave];
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    const int64_t mt = (p.M + kStreamRows - 1) / kStreamRows;
    const int64_t o0 = blockIdx.x % mt * kStreamRows;
    const I8Tile tile = find_tile(p.offsets, p.E, p.T, 16 * NT, blockIdx.x / mt);
    if (tile.first >= tile.last) return;
    const int64_t r16 = lane & 15;
    const int64_t kq = 16 * (lane >> 4);
    const int64_t wrow = min(o0 + r16, p.M - 1);  // rows behind the last one repeat it
    const int8_t* w = p.W + tile.expert * p.w_stride + wrow * p.ldw + kq;
    const int8_t* up = w + p.M * p.ldw;
    const int8_t* x[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        int64_t r = min(tile.first + 16 * n + r16, tile.last - 1);
        if (p.order) r = p.order[r] / p.topk;
        x[n] = p.X + r * p.ldx + kq;
    }
    i32x4 acc[G][NT];
#pragma unroll
    for (int g = 0; g < G; ++g)
#pragma unroll
        for (int n = 0; n < NT; ++n) acc[g][n] = i32x4{0, 0, 0, 0};
    const int64_t steps = p.K / 64;               // whole ones
    const int64_t s1 = steps * (wave + 1) / NW;
    for (int64_t s = steps * wave / NW; s < s1; ++s) {
        const u32x4 a = *(const u32x4*)(w + 64 * s);
        u32x4 b = {0, 0, 0, 0};
        if constexpr (GATE) b = *(const u32x4*)(up + 64 * s);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const u32x4 v = *(const u32x4*)(x[n] + 64 * s);
            acc[0][n] = mfma_i8(a, v, acc[0][n]);
            if constexpr (GATE) acc[G - 1][n] = mfma_i8(b, v, acc[G - 1][n]);
        }
    }
    if (p.K % 64 != 0 && wave == NW - 1) {        // the channels behind the last whole step
        const bool in = 64 * steps + kq < p.K;
        const u32x4 none = {0, 0, 0, 0};
        const u32x4 a = in ? *(const u32x4*)(w + 64 * steps) : none;
        u32x4 b = none;
        if constexpr (GATE) b = in ? *(const u32x4*)(up + 64 * steps) : none;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const u32x4 v = in ? *(const u32x4*)(x[n] + 64 * steps) : none;
            acc[0][n] = mfma_i8(a, v, acc[0][n]);
            if constexpr (GATE) acc[G - 1][n] = mfma_i8(b, v, acc[G - 1][n]);
        }
    }
#pragma unroll
    for (int g = 0; g < G; ++g)
#pragma unroll
        for (int n = 0; n < NT; ++n) sums[wave][g][n][lane] = acc[g][n];
    __syncthreads();
    if (wave >= NT) return;
    // Wave n adds token fragment n: the lane's 4 rows of W of one row of X.
    i32x4 s[G];
#pragma unroll
    for (int g = 0; g < G; ++g) {
        s[g] = sums[0][g][wave][lane];
#pragma unroll
        for (int v = 1; v < NW; ++v) s[g] += sums[v][g][wave][lane];
    }
    const int64_t t = tile.first + 16 * wave + r16, o = o0 + 4 * (lane >> 4);
    if (t >= tile.last || o >= p.M) return;
    const float xs = p.x_scale[p.order ? p.order[t] / p.topk : t];
    f32x4 y;
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = i8_result<GATE>(p, tile.expert, min(o + i, p.M - 1), xs, s[0][i], s[G - 1][i]);
    store_y4<YF32>(p.Y, t * p.ldy + o, p.M - o, p.yvec, y);
}

template <int NT>
static hipError_t stream(const I8Product& p, bool gate, bool yf32, hipStream_t st) {
    const int64_t mt = (p.M + kStreamRows - 1) / kStreamRows;
    const int64_t tiles = p.offsets ? i8_tiles(p.T, p.E, 16 * NT) : (p.T + 16 * NT - 1) / (16 * NT);
    const int nt = NT <= 2 ? 1024 : 512;
    if (mt * tiles * nt >= (int64_t)1 << 32) return hipErrorInvalidConfiguration;
    const dim3 grid((unsigned)(mt * tiles)), block((unsigned)nt);
    if (gate) return launch_kernel(k_i8_stream<NT, true, true>, grid, block, 0, st, nullptr, nullptr, p);
    return yf32 ? launch_kernel(k_i8_stream<NT, false, true>, grid, block, 0, st, nullptr, nullptr, p)
                : launch_kernel(k_i8_stream<NT, false, false>, grid, block, 0, st, nullptr, nullptr, p);
}

size_t i8_product_ws_bytes(int64_t T, int64_t K, int64_t M) { return 0; }

bool i8_product_fits(int64_t T, int64_t M) { return (T + 15) / 16 * ((M + 15) / 16) < (int64_t)1 << 22; }

hipError_t launch_i8_product(const I8Product& q, bool yf32, void* ws, hipStream_t st) {
    I8Product p = q;
    p.yvec = (uintptr_t)p.Y % 16 == 0 && p.ldy * (yf32 ? 4 : 2) % 16 == 0;
    const bool gate = p.s_down != nullptr;
    const int64_t rows = p.offsets ? (p.T + p.E - 1) / p.E : p.T;   // of one matrix, on average
    if (rows <= 16) return stream<1>(p, gate, yf32, st);
    if (rows <= 32) return stream<2>(p, gate, yf32, st);
    return stream<4>(p, gate, yf32, st);
}

}  // namespace ttq
