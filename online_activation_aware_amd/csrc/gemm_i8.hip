// Products of 8-bit codes with scales for each row of either side:
//   Y[t][o] = x_scale[t] w_scale[o] sum_j X[t][j] W[o][j],
// the sum exact in int32 on the matrix cores (K <= 2^17), for one matrix or for
// rows sorted by expert that multiply their own expert's; optionally
//   Y[t][o] = act(g) u / s[o],  g and u the products with rows o and M + o of W.
//
// Two kernels: k_i8_stream for few rows, bound by W's bytes, and k_i8_tile, with
// tiles from 64 x 32 (bound by W's bytes as well) to 256 x 256 (bound by the matrix
// cores, their power and the LDS that feeds them).  As every sum is exact, a
// result is the same whichever computes it.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "i8.hpp"
#include "rows_i8.hpp"
#include "wave.hpp"

namespace ttq {

enum { kOutBf16, kOutF32, kOutGate, kOutSums };  // Y in bf16, in fp32, gated in fp32; sums of a part of the channels

constexpr int kStreamRows = 16;                   // rows of W a workgroup
constexpr int kXcdRows = 8;                       // tiles of W a group

// W streamed once per tile of 16 NT rows of X, straight into registers: a
// workgroup owns 16 rows of W (16 of gate and of up), its NW waves share out the
// channels and add their sums through LDS.  A wave requests U steps of 64
// channels of W and X together before the first product.
template <int NT, int NW, int OUT>
__global__ __launch_bounds__(NW * kWave) void k_i8_stream(I8Product p) {
    constexpr bool GATE = OUT == kOutGate, YF32 = OUT != kOutBf16;
    constexpr int G = GATE ? 2 : 1, U = NT == 1 ? 8 / G : 4 / G;
    __shared__ i32x4 sums[NW][G][NT][kWave];
    const int lane = threadIdx.x & (kWave - 1), wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int mt = (int)((p.M + kStreamRows - 1) / kStreamRows);
    I8Tile tile{0, (int)blockIdx.x / mt * 16 * NT, 0, (int)blockIdx.x % mt};
    tile.last = min(tile.first + 16 * NT, (int)p.T);
    if (p.offsets) tile = find_tile(p.offsets, p.E, 16 * NT, mt, blockIdx.x);
    if (tile.first >= tile.last) return;
    const int64_t o0 = (int64_t)tile.mtile * kStreamRows;
    const int r16 = lane & 15, kq = 16 * (lane >> 4);
    const int64_t wrow = min(o0 + r16, p.M - 1);  // rows behind the last one repeat it
    const int8_t* w[G];
    w[0] = p.W + tile.expert * p.w_stride + wrow * p.ldw + kq;
    if constexpr (GATE) w[1] = w[0] + p.M * p.ldw;
    const int8_t* x[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        int64_t r = min(tile.first + 16 * n + r16, tile.last - 1);
        if (p.order) r = p.order[r] / p.topk;
        x[n] = p.X + r * p.ldx + kq;
    }
    // The scales of the results of waves that add, requested ahead.
    float xs = 0.f;
    I8Results<GATE> ws;
    if (wave < NT) {
        const int t = min(tile.first + 16 * wave + r16, tile.last - 1);
        xs = p.x_scale[p.order ? p.order[t] / p.topk : t];
#pragma unroll
        for (int i = 0; i < 4; ++i) ws.set(i, i8_scales<GATE>(p, tile.expert, min(o0 + 4 * (lane >> 4) + i, p.M - 1)));
    }
    i32x4 acc[G][NT];
#pragma unroll
    for (int g = 0; g < G; ++g)
#pragma unroll
        for (int n = 0; n < NT; ++n) acc[g][n] = i32x4{0, 0, 0, 0};
    const int steps = (int)(p.K / 64);            // whole ones
    const int s1 = steps * (wave + 1) / NW;
    auto batch = [&](int s, auto count) __attribute__((always_inline)) {
        constexpr int C = decltype(count)::value;
        u32x4 a[C][G], b[C][NT];
#pragma unroll
        for (int u = 0; u < C; ++u)
#pragma unroll
            for (int g = 0; g < G; ++g) a[u][g] = *(const u32x4*)(w[g] + 64 * (int64_t)(s + u));
#pragma unroll
        for (int u = 0; u < C; ++u)
#pragma unroll
            for (int n = 0; n < NT; ++n) b[u][n] = *(const u32x4*)(x[n] + 64 * (int64_t)(s + u));
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int u = 0; u < C; ++u)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int g = 0; g < G; ++g) acc[g][n] = mfma_i8(a[u][g], b[u][n], acc[g][n]);
    };
    int s = steps * wave / NW;
    for (; s + U <= s1; s += U) batch(s, std::integral_constant<int, U>{});
    for (; s < s1; ++s) batch(s, std::integral_constant<int, 1>{});
    if (p.K % 64 != 0 && wave == NW - 1) {        // the channels behind the last whole step
        const bool in = 64 * steps + kq < p.K;
        const u32x4 none = {0, 0, 0, 0};
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const u32x4 v = in ? *(const u32x4*)(x[n] + 64 * (int64_t)steps) : none;
#pragma unroll
            for (int g = 0; g < G; ++g)
                acc[g][n] = mfma_i8(in ? *(const u32x4*)(w[g] + 64 * (int64_t)steps) : none, v, acc[g][n]);
        }
    }
#pragma unroll
    for (int g = 0; g < G; ++g)
#pragma unroll
        for (int n = 0; n < NT; ++n) sums[wave][g][n][lane] = acc[g][n];
    __syncthreads();
    if (wave >= NT) return;
    // Wave n adds token fragment n: the lane's 4 rows of W of one row of X.
    i32x4 t4[G];
#pragma unroll
    for (int g = 0; g < G; ++g) {
        t4[g] = sums[0][g][wave][lane];
#pragma unroll
        for (int v = 1; v < NW; ++v) t4[g] += sums[v][g][wave][lane];
    }
    const int64_t t = tile.first + 16 * wave + r16, o = o0 + 4 * (lane >> 4);
    if (t >= tile.last || o >= p.M) return;
    ws.ready();
    store_y4<YF32>(p.Y, t * p.ldy + o, p.M - o, p.yvec, ws.of(p.act, xs, t4[0], t4[G - 1]));
}

template <int NT, int NW>
static hipError_t stream(const I8Product& p, int out, hipStream_t st) {
    const int64_t mt = (p.M + kStreamRows - 1) / kStreamRows;
    const int64_t blocks = p.offsets ? i8_blocks(p.T, p.E, 16 * NT, mt) : mt * ((p.T + 16 * NT - 1) / (16 * NT));
    const dim3 grid((unsigned)blocks), block(NW * kWave);
    if (out == kOutGate) return launch_kernel(k_i8_stream<NT, NW, kOutGate>, grid, block, 0, st, nullptr, nullptr, p);
    return out == kOutF32 ? launch_kernel(k_i8_stream<NT, NW, kOutF32>, grid, block, 0, st, nullptr, nullptr, p)
                          : launch_kernel(k_i8_stream<NT, NW, kOutBf16>, grid, block, 0, st, nullptr, nullptr, p);
}

// One token whose row is quantized on the way, in one launch: every workgroup
// forms the codes itself, in LDS, the token's values requested first and its own
// first codes of W behind them.  Its waves take `blocks` blocks of 16 rows of W
// at a time and share out the channels of each.  (14336 -> 4096: k_quantize_rows
// and k_i8_stream take 5 and 12 us one after the other, this 12 to 14: W's bytes at
// 4.5 TB/s.)
constexpr int kOneWaves = 16, kOneSegs = 2;       // vectors of eight values a lane holds
__host__ __device__ constexpr int one_pad(int64_t K) { return (int)((K + 63) / 64 * 64); }

template <bool XF32, bool DIV, bool YF32>
__global__ __launch_bounds__(kOneWaves * kWave) void k_i8_one(I8RowsArgs x, I8Product p, int blocks,
                                                                int share, int turns) {
    constexpr int NT = kOneWaves * kWave, U = 4;
    __shared__ i32x4 sums[kOneWaves][kWave];
    uint32_t* part = (uint32_t*)sums;             // of the waves' maxima
    extern __shared__ __attribute__((aligned(16))) int8_t codes[];   // [kp + 64], zeros from channel K on
    const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int K = (int)p.K, kp = one_pad(K), r16 = lane & 15, kq = 16 * (lane >> 4);
    const int wb = wave / share, wk = wave % share;   // this wave's block, its place among the `share` waves of it
    const int steps = kp / 64, s0 = steps * wk / share, s1 = steps * (wk + 1) / share;
    const int last = max(s1 - 1, 0);              // (a wave may have no step)

    RowScale<DIV ? 1 : 0> s[kOneSegs];            // (divisions: a reciprocal of one use costs more)
    RowVector<XF32> y[kOneSegs];                  // (lanes behind the last channel repeat it)
#pragma unroll
    for (int u = 0; u < kOneSegs; ++u) {
        const int k = min((u * NT + tid) * kRowSeg, K - kRowSeg);
        y[u].load(x.X, k);
        s[u].load(x.s + k);
    }
    f32x4 ws;                                     // of the turn's outputs
    auto load_ws = [&](int turn) __attribute__((always_inline)) {
        const int64_t o = (int64_t)(turn * blocks + wb) * kStreamRows + 4 * (lane >> 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) ws[i] = p.w_scale[min(o + i, p.M - 1)];
    };
    load_ws(blockIdx.x);
    const int8_t* w;
    auto rows_of = [&](int turn) __attribute__((always_inline)) {
        return p.W + min((int64_t)(turn * blocks + wb) * kStreamRows + r16, p.M - 1) * p.ldw;   // rows behind the last one repeat it
    };
    // U steps of this wave's rows of W from step s on; behind the wave's last step,
    // and behind the last channel, any codes: the token's are zero there.
    auto fetch = [&](u32x4 (&a)[U], int s) __attribute__((always_inline)) {
#pragma unroll
        for (int u = 0; u < U; ++u) a[u] = *(const u32x4*)(w + min(64 * min(s + u, last) + kq, K - 16));
    };
    u32x4 a[2][U];
    w = rows_of(blockIdx.x);
    fetch(a[0], s0);
    fetch(a[1], s0 + U);
    __builtin_amdgcn_sched_barrier(0);

    float v[kOneSegs][kRowSeg];
    uint32_t top = 0;
#pragma unroll
    for (int u = 0; u < kOneSegs; ++u) {
#pragma unroll
        for (int c = 0; c < kRowSeg; ++c) v[u][c] = DIV ? y[u][c] / s[u].s[DIV ? c : 0] : y[u][c];
        top = row_top(v[u], top);
    }
    top = wave_max_u32(top);
    if (lane == 0) part[wave] = top;
    __syncthreads();
#pragma unroll
    for (int n = 0; n < kOneWaves; ++n) top = max(top, part[n]);
    const float xs = row_scale(top);
#pragma unroll
    for (int u = 0; u < kOneSegs; ++u) {
        const int k = (u * NT + tid) * kRowSeg;
        if (k < K) *(u32x2*)(codes + k) = row_codes(v[u], xs);
    }
    if (tid < kp + 64 - K) codes[K + tid] = 0;
    __syncthreads();

#pragma unroll 1
    for (int g = blockIdx.x; g < turns; g += gridDim.x) {
        const int64_t o = (int64_t)(g * blocks + wb) * kStreamRows + 4 * (lane >> 4);
        i32x4 acc = {0, 0, 0, 0};
        auto multiply = [&](const u32x4 (&f)[U], int s) __attribute__((always_inline)) {
#pragma unroll
            for (int u = 0; u < U; ++u)
                acc = mfma_i8(f[u], *(const u32x4*)(codes + (s + u < s1 ? 64 * (s + u) : kp) + kq), acc);
        };
#pragma unroll 1
        for (int s = s0; s < s1; s += 2 * U) {
            multiply(a[0], s);
            if (s + 2 * U < s1) fetch(a[0], s + 2 * U);
            multiply(a[1], s + U);
            if (s + 3 * U < s1) fetch(a[1], s + 3 * U);
        }
        if (g + gridDim.x < turns) {              // the next turn's first codes
            w = rows_of(g + gridDim.x);
            fetch(a[0], s0);
            fetch(a[1], s0 + U);
        }
        sums[wave][lane] = acc;
        __syncthreads();
        if (wk == 0 && r16 == 0 && o < p.M) {     // (all columns are the token's)
            for (int n = 1; n < share; ++n) acc += sums[wave + n][lane];
            f32x4 r;
#pragma unroll
            for (int i = 0; i < 4; ++i) r[i] = (float)acc[i] * xs * ws[i];
            load_ws(g + gridDim.x);
            store_y4<YF32>(p.Y, o, p.M - o, p.yvec, r);
        }
        __syncthreads();
    }
}

// (33 KB of LDS at most.)
bool i8_one_fits(int64_t T, int64_t K) { return T == 1 && K <= kOneWaves * kWave * kRowSeg * kOneSegs; }

hipError_t launch_i8_one(const I8RowsArgs& x, const I8Product& q, bool yf32, hipStream_t st) {
    I8Product p = q;
    p.yvec = (uintptr_t)p.Y % 16 == 0;
    // One workgroup a compute unit, so that each quantizes once for its turns;
    // more blocks a turn where rows of W allow it, so that a wave has more steps.
    const int64_t groups = (p.M + kStreamRows - 1) / kStreamRows;
    const int blocks = groups >= 768 ? 4 : groups >= 384 ? 2 : 1;
    const int64_t turns = (groups + blocks - 1) / blocks;
    const dim3 grid((unsigned)std::min<int64_t>(turns, 256)), block(kOneWaves * kWave);
    const size_t lds = (size_t)one_pad(p.K) + 64;
#define TTQ_ONE(XF, DV)                                                                                             \
    do {                                                                                                            \
        if (yf32) return launch_kernel(k_i8_one<XF, DV, true>, grid, block, lds, st, nullptr, nullptr, x, p, blocks,       \
                                                         kOneWaves / blocks, (int)turns);                                    \
        return launch_kernel(k_i8_one<XF, DV, false>, grid, block, lds, st, nullptr, nullptr, x, p, blocks,              \
                             kOneWaves / blocks, (int)turns);                                                                \
    } while (0)
    if (x.xf32) {
        if (x.s) TTQ_ONE(true, true);
        TTQ_ONE(true, false);
    }
    if (x.s) TTQ_ONE(false, true);
    TTQ_ONE(false, false);
#undef TTQ_ONE
}

// Tiles of BM rows of W x BN rows of X, WM x WN waves.  Both operands arrive by
// buffer -> LDS DMA, 128 channels (a line) a row and step, in two slots; an LDS
// row's 16-byte chunks are exclusive-or'ed with its number (conflict-free).
//
// A step has two phases: X and the first half of every wave's rows of W, then the
// second half; each part of a slot is requested again as soon as every wave has
// read it, three phases ahead of its use.  (A step's 64 KB take longer than one
// step's products to arrive.  A third slot of W for the smaller tiles: 64 x 4096 ->
// 14336 15.1 us, two 14.5; 768 rows 55 and 54.)  Of 256 x 256: 8192 rows of 4096 ->
// 4096 in 115 to 130 us, 2.1 to 2.4 POP/s, the matrix pipes busy for 55% of the
// cycles; with all codes zero 100 us, so that power sets a part of it.
template <int BM, int BN, int WM, int WN, int OUT>
__global__ __launch_bounds__(WM * WN * kWave, 1) void k_i8_tile(I8Product p) {
    constexpr bool GATE = OUT == kOutGate, YF32 = OUT != kOutBf16;
    constexpr int NW = WM * WN;
    constexpr int FA = BM / WM / 16, FB = BN / WN / 16;         // fragments of 16 rows per wave
    constexpr int HR = BM / WM / 2;                             // a wave's rows of W a phase
    constexpr int XOPS = BN * kLdsRowB / 1024 / NW, WOPS = BM / 2 * kLdsRowB / 1024 / NW;   // DMA operations of 1 KB per wave
    constexpr int G = GATE ? 2 : 1, BO = BM / G;                // outputs of a tile
    constexpr int SW = BM * kLdsRowB, SX = BN * kLdsRowB;       // slots: W of the first phase and of the second; X
    constexpr int kStep = kLdsRowB;
    __shared__ __attribute__((aligned(1024))) uint8_t lds[2 * SW + 2 * SX];
    const int lane = threadIdx.x & (kWave - 1), wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int wm = wave % WM, wn = wave / WM;
    // One matrix: the workgroups that an XCD receives are consecutive in an order
    // that walks groups of kXcdRows tiles of W across the tiles of X, so that its L2
    // holds what they share.
    const int mt = (int)((p.M + BO - 1) / BO), n = (int)gridDim.x / p.splits;
    const int part = OUT == kOutSums ? (int)blockIdx.x / n : 0, bx = (int)blockIdx.x - part * n;
    I8Tile tile;
    if (p.offsets) {
        tile = find_tile(p.offsets, p.E, BN, mt, bx);
    } else {
        const int x = bx % 8, v = x * (n / 8) + min(x, n % 8) + bx / 8, nt = n / mt;
        const int g0 = v / (kXcdRows * nt) * kXcdRows, gw = min(kXcdRows, mt - g0), in = v - g0 * nt;
        const int first = in / gw * BN;
        tile = {0, first, min(first + BN, (int)p.T), g0 + in % gw};
    }
    const int rows = tile.last - tile.first;
    if (rows <= 0) return;
    const int64_t o0 = (int64_t)tile.mtile * BO;
    const int8_t* W = p.W + tile.expert * p.w_stride + o0 * p.ldw;
    const int64_t wrows = GATE ? 2 * p.M - o0 : min((int64_t)BM, p.M - o0);
    const rsrc_t rw = make_rsrc(W, (wrows - 1) * p.ldw + p.K);
    const int8_t* X = p.X + (p.order ? 0 : (int64_t)tile.first * p.ldx);
    const rsrc_t rx = make_rsrc(X, ((p.order ? p.xrows : rows) - 1) * p.ldx + p.K);

    // A DMA operation fills eight LDS rows; lane l lands in row l / 8 of them at
    // position l % 8, holding chunk (l % 8) ^ (row & 7).
    const int rl = lane >> 3, ch = (lane & 7) ^ rl;
    int xoff[XOPS], woff[2][WOPS];
#pragma unroll
    for (int i = 0; i < XOPS; ++i) {
        const int r = 8 * (XOPS * wave + i) + rl;
        const int src = r >= rows ? 0 : p.order ? p.order[tile.first + r] / p.topk : r;
        xoff[i] = r >= rows ? INT32_MIN : src * (int)p.ldx + 16 * ch;   // behind the last row: zeros, not read
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < WOPS; ++i) {
            const int l = 8 * (WOPS * wave + i) + rl, w = l / HR * 2 * HR + h * HR + l % HR;
            // Gate and up: 16 rows of either in turn.
            const int r = GATE ? (w >> 5) * 16 + (w & 15) + ((w >> 4) & 1) * (int)p.M : w;
            woff[h][i] = r * (int)p.ldw + 16 * ch;
        }
    i32x4 acc[FA][FB];
#pragma unroll
    for (int i = 0; i < FA; ++i)
#pragma unroll
        for (int j = 0; j < FB; ++j) acc[i][j] = i32x4{0, 0, 0, 0};

    int nk = (int)((p.K + kStep - 1) / kStep), k0 = 0;
    if constexpr (OUT == kOutSums) {              // this part's steps
        k0 = nk * part / p.splits;
        nk = nk * (part + 1) / p.splits;
    }
    auto issue_w = [&](int slot, int k, int h) __attribute__((always_inline)) {
        const int none = k >= nk ? INT32_MIN : 0; // behind the last step: not read
#pragma unroll
        for (int i = 0; i < WOPS; ++i)
            dma_to_lds<16>(rw, lds + slot + h * (SW / 2) + (wave * WOPS + i) * 1024, woff[h][i] | none, k * kStep);
    };
    auto issue_x = [&](int slot, int k) __attribute__((always_inline)) {
        // Behind the last channel X is zero: an offset past the descriptor.
        const int gone = k >= nk || 16 * ch >= (int)p.K - k * kStep ? INT32_MIN : 0;
#pragma unroll
        for (int i = 0; i < XOPS; ++i)
            dma_to_lds<16>(rx, lds + 2 * SW + slot + (wave * XOPS + i) * 1024, xoff[i] | gone, k * kStep);
    };
    u32x4 a[2][FA / 2], b[2][FB];                 // fragments of the two 64-channel halves
    const int off[2] = {lds_swz(lane & 15, lane >> 4), lds_swz(lane & 15, 4 + (lane >> 4))};
    const int wread = wm * HR * kLdsRowB, xread = 2 * SW + wn * 16 * kLdsRowB;
    // The fragments of X are dealt out to the waves one by one: a tile with fewer
    // rows has fewer products in every wave (fb of them a fragment of W).
    const int frags = (rows + 15) / 16, fb = GATE || o0 + wm * FA * 16 < p.M ? max((frags - wn + WN - 1) / WN, 0) : 0;
    auto phase = [&](int wslot, int xslot, int h, auto count) __attribute__((always_inline)) {
        constexpr int NB = decltype(count)::value;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const uint8_t* from = lds + off[s] + wslot + wread + h * (SW / 2);
            const uint8_t* x = lds + off[s] + xslot + xread;
            if (h == 0)
#pragma unroll
                for (int j = 0; j < NB; ++j) b[s][j] = *(const u32x4*)(x + j * WN * 16 * kLdsRowB);
#pragma unroll
            for (int i = 0; i < FA / 2; ++i) a[s][i] = *(const u32x4*)(from + i * 16 * kLdsRowB);
        }
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int i = 0; i < FA / 2; ++i)
#pragma unroll
                for (int j = 0; j < NB; ++j)
                    acc[h * (FA / 2) + i][j] = mfma_i8(a[s][i], b[s][j], acc[h * (FA / 2) + i][j]);
    };
    // In the order of the steps: the parts that step 0 finds requested.
    issue_x(0, k0);
    issue_w(0, k0, 0);
    issue_w(0, k0, 1);
    issue_x(SX, k0 + 1);
    issue_w(SW, k0 + 1, 0);
    // The tile's scales, a thread one of either side: through LDS to their lanes
    // once the products are done.  (Other LDS arrays, or stores to this one before
    // the loop, make the compiler wait for every DMA before a fragment is read.)
    static_assert(BN <= NW * kWave && BO <= NW * kWave, "a thread holds one scale of either side");
    const int ts = tile.first + min((int)threadIdx.x, rows - 1);
    const float xs = p.x_scale[p.order ? p.order[ts] / p.topk : ts];
    const I8Scales<GATE> wscale = i8_scales<GATE>(p, tile.expert, min(o0 + threadIdx.x, p.M - 1));
    // Operations requested after the parts that the next phase needs.
    constexpr int kLater = 2 * WOPS + XOPS;
    wait_vmcnt<kLater>();
    sync_lds();
    int wcur = 0, xcur = 0;
    auto steps = [&](auto count) __attribute__((always_inline)) {
        constexpr bool kWork = decltype(count)::value > 0;
        for (int k = k0; k < nk; ++k) {
            issue_w(SW - wcur, k + 1, 1);
            if constexpr (kWork) phase(wcur, xcur, 0, count);
            wait_vmcnt<kLater>();
            sync_lds();
            issue_x(xcur, k + 2);
            issue_w(wcur, k + 2, 0);
            if constexpr (kWork) phase(wcur, xcur, 1, count);
            wait_vmcnt<kLater>();
            sync_lds();
            wcur = SW - wcur;
            xcur = SX - xcur;
        }
    };
    if (fb == FB) steps(std::integral_constant<int, FB>{});
    else if (FB > 3 && fb == 3) steps(std::integral_constant<int, FB < 3 ? FB : 3>{});
    else if (FB > 2 && fb == 2) steps(std::integral_constant<int, FB < 2 ? FB : 2>{});
    else if (fb == 1) steps(std::integral_constant<int, 1>{});
    else steps(std::integral_constant<int, 0>{});
    wait_vmcnt<0>();

    if constexpr (OUT == kOutSums) {              // [parts][T][mp] int32, added by k_i8_sum
        const int64_t mp = (p.M + 3) / 4 * 4;
        int* out = p.sums + (int64_t)part * p.T * mp;
#pragma unroll
        for (int i = 0; i < FA; ++i) {
            const int64_t o = o0 + (wm * FA + i) * 16 + 4 * (lane >> 4);
#pragma unroll
            for (int j = 0; j < FB; ++j) {
                const int tl = (j * WN + wn) * 16 + (lane & 15);
                if (tl < rows && o < p.M) *(i32x4*)(out + (int64_t)(tile.first + tl) * mp + o) = acc[i][j];
            }
        }
        return;
    }
    // Each wave has waited for its own DMA.  That behind the last step writes zeros
    // where the scales go (one slot or the other, by the number of steps), so that
    // they are stored when every wave has.
    sync_lds();
    float *sx = (float*)lds, *sw = sx + BN;
    if (threadIdx.x < BN) sx[threadIdx.x] = xs;
    if (threadIdx.x < BO) {
        sw[threadIdx.x] = wscale.g;
        if constexpr (GATE) {
            sw[BO + threadIdx.x] = wscale.u;
            sw[2 * BO + threadIdx.x] = wscale.s;
        }
    }
    __syncthreads();
    if (fb == 0) return;
    // The lane's 4 consecutive outputs of a row of X, for each pair of fragments.
    const bool whole = rows == BN && o0 + BO <= p.M && p.yvec;
#pragma unroll
    for (int i = 0; i < FA; i += G) {
        const int ol = (wm * FA + i) * (16 / G) + 4 * (lane >> 4);
        const int64_t o = o0 + ol;
        I8Results<GATE> w;
        w.g = *(const f32x4*)(sw + ol);
        if constexpr (GATE) {
            w.u = *(const f32x4*)(sw + BO + ol);
            w.s = *(const f32x4*)(sw + 2 * BO + ol);
        }
        w.ready();
#pragma unroll
        for (int j = 0; j < FB; ++j) {
            const int tl = (j * WN + wn) * 16 + (lane & 15);
            const float xt = sx[tl];
            const f32x4 y = w.of(p.act, xt, acc[i][j], acc[i + G - 1][j]);
            const int64_t at = (int64_t)(tile.first + tl) * p.ldy + o;
            if (whole) store_y4<YF32>(p.Y, at, 4, 1, y);
            else if (tl < rows && o < p.M) store_y4<YF32>(p.Y, at, p.M - o, p.yvec, y);
        }
    }
}

// Y from the parts' sums, added exactly in int32.
template <bool YF32>
__global__ __launch_bounds__(256) void k_i8_sum(I8Product p) {
    const int64_t quads = (p.M + 3) / 4, all = p.T * quads;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < all; i += (int64_t)gridDim.x * 256) {
        const int64_t t = i / quads, o = (i - t * quads) * 4;
        i32x4 s = {0, 0, 0, 0};
        for (int c = 0; c < p.splits; ++c) s += *(const i32x4*)(p.sums + (c * all + i) * 4);
        I8Results<false> w;
#pragma unroll
        for (int r = 0; r < 4; ++r) w.set(r, i8_scales<false>(p, 0, min(o + r, p.M - 1)));
        store_y4<YF32>(p.Y, t * p.ldy + o, p.M - o, p.yvec, w.of(0, p.x_scale[t], s, s));
    }
}

template <int BM, int BN, int WM, int WN>
static hipError_t tiled(const I8Product& p, int out, hipStream_t st) {
    const bool gate = out == kOutGate, yf32 = out == kOutF32;
    const int64_t bo = gate ? BM / 2 : BM, mt = (p.M + bo - 1) / bo;
    const int64_t blocks = p.offsets ? i8_blocks(p.T, p.E, BN, mt) : mt * ((p.T + BN - 1) / BN);
    const dim3 grid((unsigned)(blocks * p.splits)), block(WM * WN * kWave);
    if (p.splits > 1) {
        const hipError_t e = launch_kernel(k_i8_tile<BM, BN, WM, WN, kOutSums>, grid, block, 0, st, nullptr, nullptr, p);
        if (e != hipSuccess) return e;
        const int64_t work = p.T * ((p.M + 3) / 4);
        const dim3 sum((unsigned)std::min<int64_t>((work + 255) / 256, 8192));
        return yf32 ? launch_kernel(k_i8_sum<true>, sum, dim3(256), 0, st, nullptr, nullptr, p)
                    : launch_kernel(k_i8_sum<false>, sum, dim3(256), 0, st, nullptr, nullptr, p);
    }
    if (gate) return launch_kernel(k_i8_tile<BM, BN, WM, WN, kOutGate>, grid, block, 0, st, nullptr, nullptr, p);
    return yf32 ? launch_kernel(k_i8_tile<BM, BN, WM, WN, kOutF32>, grid, block, 0, st, nullptr, nullptr, p)
                : launch_kernel(k_i8_tile<BM, BN, WM, WN, kOutBf16>, grid, block, 0, st, nullptr, nullptr, p);
}

// What a product takes by each kernel, in us, fitted to 220 shapes (1 to 8192
// rows, 256 to 14336 channels, 768 to 14336 outputs), each timed with every
// kernel; the choice by these costs lies 2% over the best kernel of each shape on
// average, a third at most.  Some of them (us): 8192 rows of 4096 -> 4096: 256 x
// 256 124, 256 x 128 153, 128 x 64 193; 2048: 56, 40, 52; 512: 57, 31, 18, 64 x 32
// 20; 64: 64 x 32 12, streamed 14; 16: 12 and 7; 14336 -> 4096, 1024 rows: 256 x 128
// in two parts 74, in one 103; 64 rows: 128 x 64 in eight parts 21, in one 48.  (What their
// bytes or products take: 4096 -> 4096, 8192 rows 131 at the library's rate, 2048 33, 512
// 8.2, 64 3.4; 14336 -> 4096, 1024 rows 57, 64 rows 12.)
//
// A tile takes `start` and for each 128 channels `step`, `full` where every
// compute unit has a tile and `more` for each further one that it works on at the
// same time, at most `fit`.  Parts of the channels cost a second launch and the
// traffic of their sums.  Nothing is faster than W's bytes.
struct I8Kernel {
    int bm, bn, threads, fit;
    double start, step, full, more;
};
constexpr I8Kernel kTiles[] = {{64, 32, 128, 5, 3.1, 0.29, 0.25, 0.14},
                               {128, 64, 256, 3, 3.7, 0.51, 0.44, 0.31},
                               {256, 128, 512, 1, 5.3, 0.67, 0.95, 0},
                               {256, 256, 512, 1, 8.5, 0.67, 1.52, 0}};
constexpr int kMaxSplits = 16;

struct I8Choice {
    int kernel;                                   // of kTiles; -1, -2: streamed for tiles of 16, 32 rows
    int splits;
};

// A grid has fewer than 2^32 threads.
static bool grid_fits(double blocks, int threads) { return blocks * threads < 4294967296.0; }

// Workgroups of tiles of `rows` x `outputs` of T x M: for one matrix (E == 0), or at
// most for E (i8_blocks).
static double grid_blocks(int64_t T, int64_t M, int64_t E, int64_t rows, int64_t outputs) {
    if (E == 0) return (double)((T + rows - 1) / rows) * (double)((M + outputs - 1) / outputs);
    return ((double)(T / rows) + 1 + (double)E) * ((double)(M / outputs) + 8);
}

// The largest tiles cover T x M.
bool i8_product_fits(int64_t T, int64_t M, int64_t E) { return grid_fits(grid_blocks(T, M, E, 256, E == 0 ? 256 : 128), 512); }

static I8Choice choose(int64_t T, int64_t K, int64_t M, int64_t E, bool experts, bool gate) {
    const int64_t rows = experts ? std::max<int64_t>((T + E - 1) / E, 1) : T;    // of a matrix, on average
    const double mats = experts ? (double)std::min(T, E) : 1;
    const double steps = (double)((K + kLdsRowB - 1) / kLdsRowB), codes = mats * (double)(K * M) * (gate ? 2 : 1) / 1e6;
    I8Choice best{3, 1};                          // (its grid fits)
    double least = 0;
    auto offer = [&](double us, int kernel, int splits) {
        us = std::max(us, 3.1 + codes / 5.2 + (splits > 1 ? 3.2 : 0.0));
        if (least > 0 && us >= least) return;
        least = us;
        best = {kernel, splits};
    };
    for (int k = 0; k < 4; ++k) {
        const I8Kernel& c = kTiles[k];
        const int64_t bo = gate ? c.bm / 2 : c.bm;
        for (int s = 1; s <= (experts ? 1 : kMaxSplits); s *= 2) {
            if (s > 1 && steps < 2 * s) break;
            const double tiles = (double)(((M + bo - 1) / bo) * ((rows + c.bn - 1) / c.bn) * s) * mats;
            if (!grid_fits(grid_blocks(T, M, experts ? E : 0, c.bn, bo) * s, c.threads)) break;
            const double n = std::ceil(tiles / 256), at_once = std::min(n, (double)c.fit);
            const double step = c.step + (c.full - c.step) * std::min(tiles / 256, 1.0) + c.more * (at_once - 1);
            offer(n / at_once * (c.start + steps / s * step) +
                      (s > 1 ? 3.2 + (double)(s + 1) * T * M * 4 / 3.1e6 : 0.0), k, s);
        }
    }
    for (int nt = 1; nt <= 2 && rows <= 128; ++nt) {
        const double tiles = (double)((rows + 16 * nt - 1) / (16 * nt));
        const double x = codes * tiles * std::min<double>(rows, 16 * nt) / 16;
        if (!grid_fits(grid_blocks(T, M, experts ? E : 0, 16 * nt, kStreamRows), 256)) break;
        offer(3.0 + codes / 8.6 + 0.119 * x + 0.9 * K / 4096 + (nt - 1) * (0.03 + 5e-6 * M * tiles), -nt, 1);
    }
    return best;
}

size_t i8_product_ws_bytes(int64_t T, int64_t K, int64_t M) {
    const I8Choice c = choose(T, K, M, 1, false, false);
    return c.splits > 1 ? (size_t)c.splits * T * ((M + 3) / 4 * 4) * 4 : 0;
}

hipError_t launch_i8_product(const I8Product& q, bool yf32, void* ws, hipStream_t st) {
    I8Product p = q;
    p.yvec = (uintptr_t)p.Y % 16 == 0 && p.ldy * (yf32 ? 4 : 2) % 16 == 0;
    const int out = p.s_down != nullptr ? kOutGate : yf32 ? kOutF32 : kOutBf16;
    const I8Choice c = choose(p.T, p.K, p.M, p.E, p.offsets != nullptr, out == kOutGate);
    p.splits = c.splits;
    p.sums = (int*)ws;
    switch (c.kernel) {
        case 0: return tiled<64, 32, 2, 1>(p, out, st);
        case 1: return tiled<128, 64, 2, 2>(p, out, st);
        case 2: return tiled<256, 128, 2, 4>(p, out, st);
        case 3: return tiled<256, 256, 2, 4>(p, out, st);
        case -1: return stream<1, 4>(p, out, st);
    }
    return stream<2, 4>(p, out, st);
}

}  // namespace ttq
