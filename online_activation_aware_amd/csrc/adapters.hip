// Low-rank adapters of many requests at once:
//   Y[t] = C[t] + scale_a B_a (A_a x_t),   a = ids[t],
// where A_a is the adapter's first r_a rows of [rank][K], B_a the first r_a
// columns of [M][rank]; a token whose id names no adapter gets C[t] itself.
//
// Two launches: z[t][k] = sum_j A[a][k][j] x[t][j] (fp32, into the
// workspace), then Y.
#include "common.hpp"
#include "launch.hpp"

namespace ttq {

template <bool F32>
__device__ __forceinline__ float ld_val(const void* p, int64_t i) {
    if constexpr (F32) return ((const float*)p)[i];
    else return bf16_to_f32(((const uint16_t*)p)[i]);
}

// Rows of adapter a in use; 0 where the id names none.
__device__ __forceinline__ int adapter_rank(const AdapterTable& ad, int a) {
    if (a < 0 || a >= ad.n) return 0;
    if (ad.ranks == nullptr) return ad.rank;
    const int r = ad.ranks[a];
    return r < 0 ? 0 : r > ad.rank ? ad.rank : r;
}

// One workgroup per token; wave w takes ranks w, w + 4, ...
template <bool XF32, bool AF32>
__global__ __launch_bounds__(256) void k_adapter_z(const void* __restrict__ X, int64_t K, int64_t ldx, AdapterTable ad,
                                                   float* __restrict__ Z) {
    const int64_t t = blockIdx.x;
    const int lane = threadIdx.x & (kWave - 1);
    const int a = ad.ids[t];
    const int r = adapter_rank(ad, a);
    for (int k = threadIdx.x / kWave; k < r; k += 4) {
        float acc = 0.f;
        for (int64_t j = lane; j < K; j += kWave)
            acc = __builtin_fmaf(ld_val<AF32>(ad.A, ((int64_t)a * ad.rank + k) * K + j), ld_val<XF32>(X, t * ldx + j), acc);
#pragma unroll
        for (int s = 1; s < kWave; s <<= 1) acc += __shfl_xor(acc, s);
        if (lane == 0) Z[t * ad.rank + k] = acc;
    }
}

template <bool CF32, bool AF32, bool YF32>
__global__ __launch_bounds__(256) void k_adapter_y(const float* __restrict__ Z, AdapterTable ad, const void* C,
                                                   int64_t ldc, int64_t M, void* Y, int64_t ldy) {
    const int64_t t = blockIdx.x;
    const int a = ad.ids[t];
    const int r = adapter_rank(ad, a);
    for (int64_t o = (int64_t)blockIdx.y * 256 + threadIdx.x; o < M; o += (int64_t)gridDim.y * 256) {
    float acc = 0.f;
    for (int k = 0; k < r; ++k)
        acc = __builtin_fmaf(ld_val<AF32>(ad.B, ((int64_t)a * M + o) * ad.rank + k), Z[t * ad.rank + k], acc);
    if (r > 0 && ad.scale != nullptr) acc *= ad.scale[a];
    const float c = C ? ld_val<CF32>(C, t * ldc + o) : 0.f;
    const float y = r > 0 ? c + acc : c;
    if constexpr (YF32) ((float*)Y)[t * ldy + o] = y;
    else ((uint16_t*)Y)[t * ldy + o] = (uint16_t)f32_to_bf16(y);
    }
}

size_t adapters_ws_bytes(int64_t T, int64_t K, int rank) { return (size_t)T * rank * 4; }

hipError_t launch_adapters(const void* X, bool xf32, int64_t T, int64_t K, int64_t ldx, const AdapterTable& ad,
                           const void* C, bool cf32, int64_t ldc, int64_t M, void* Y, bool yf32, int64_t ldy, float* Z,
                           hipStream_t st) {
#define TTQ_AZ(XF, AF) \
    e = launch_kernel(k_adapter_z<XF, AF>, dim3((unsigned)T), dim3(256), 0, st, nullptr, nullptr, X, K, ldx, ad, Z)
    hipError_t e;
    if (xf32) { if (ad.f32) TTQ_AZ(true, true); else TTQ_AZ(true, false); }
    else { if (ad.f32) TTQ_AZ(false, true); else TTQ_AZ(false, false); }
#undef TTQ_AZ
    if (e != hipSuccess) return e;
    const dim3 grid((unsigned)T, (unsigned)((M + 255) / 256 < 65535 ? (M + 255) / 256 : 65535));
#define TTQ_AY(CF, AF, YF)                                                                                       \
    return launch_kernel(k_adapter_y<CF, AF, YF>, grid, dim3(256), 0, st, nullptr, nullptr, (const float*)Z, ad, \
                         C, ldc, M, Y, ldy)
    if (cf32) {
        if (ad.f32) { if (yf32) TTQ_AY(true, true, true); else TTQ_AY(true, true, false); }
        else { if (yf32) TTQ_AY(true, false, true); else TTQ_AY(true, false, false); }
    }
    if (ad.f32) { if (yf32) TTQ_AY(false, true, true); else TTQ_AY(false, true, false); }
    if (yf32) TTQ_AY(false, false, true); else TTQ_AY(false, false, false);
#undef TTQ_AY
}

}  // namespace ttq
