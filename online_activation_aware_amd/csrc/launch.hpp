// Kernel launchers (host side) used by the C ABI in ttq_api.cpp.
#pragma once

#include <hip/hip_ext.h>
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ttq.h"

namespace ttq {

// Stage timing: the first kernel of a stage records `start` as it starts and
// the last records `stop` as it ends (hipExtLaunchKernel stamps the dispatch
// itself, so nothing extra is enqueued).  Null events: a plain launch.
struct StageTimer {
    hipEvent_t start = nullptr;
    hipEvent_t stop = nullptr;
};

// Low-rank term added in the projection GEMM's epilogue: Y += Z B^T, fp32.
struct LowrankEpilogue {
    const float* Z;   // [nz][T][rank]: Z = the nz partials added in order
    const float* B;   // [M][rank]
    int rank;
    int nz = 1;
};

template <typename F, typename... Args>
inline hipError_t launch_kernel(F kern, dim3 grid, dim3 block, size_t lds, hipStream_t st, hipEvent_t e0,
                                hipEvent_t e1, Args... args) {
    // (The plain launch costs the host 0.4 us less than one that could stamp.)
    if (e0 == nullptr && e1 == nullptr) kern<<<grid, block, lds, st>>>(args...);
    else hipExtLaunchKernelGGL(kern, grid, block, (std::uint32_t)lds, st, e0, e1, 0u, args...);
    return hipGetLastError();
}

// K-slice split of the low-rank Z = A X pass.
int lowrank_slices(int64_t T, int64_t K, int64_t* slice_len);

// Statistics in one launch (no workspace).  bsum (optional, ceil(K/16)
// doubles): per-16-channel block sums of c = ssq / T, from which the
// quantizer forms lambda = lambda_rel * mean(c).  p: moment order of the
// statistic, sum |x|^p (2: sums of squares).
hipError_t launch_stats(const void* X, bool xf32, int64_t T, int64_t K, int64_t ldx, double* ssq,
                        int accumulate, hipStream_t st, double* bsum = nullptr, StageTimer tm = {},
                        double p = 2.0);
hipError_t launch_awq_scales(const double* ssq, int64_t n_tokens, int64_t K, float alpha,
                             float lambda_rel, float p, float* s, hipStream_t st);
// Scales evaluated inside the quantizer from the statistics (instead of a
// given s): lambda = lambda_rel * blocks_total(bsum) / K, then
// s[j] = awq_scale(ssq[j], tn, lambda, e), also stored to s_out.
struct QScaleSrc {
    const double* ssq;
    const double* bsum;
    double lambda_rel;
    double tn;
    double e;
    float* s_out;
};
hipError_t launch_quantize(const void* W, bool wf32, int64_t M, int64_t K, int64_t ldw,
                           const float* s, int bits, int group, const float* B, const float* A,
                           int rank, uint32_t* codes, uint16_t* scale, uint16_t* zero,
                           uint16_t* wq, hipStream_t st, const QScaleSrc* qs = nullptr,
                           StageTimer tm = {});
hipError_t launch_qgemm(const void* X, bool xf32, int64_t T, int64_t K, int64_t ldx,
                        const float* s, const uint32_t* codes, const uint16_t* scale,
                        const uint16_t* zero, int64_t M, int bits, int group, void* Y, bool yf32,
                        int64_t ldy, uint16_t* wq, hipStream_t st, StageTimer tm = {});
// Prompt-sized projections use the dequantized weight w~ ([M][K] bf16) and
// the matrix-core GEMM; smaller ones (and fp32 X) the fused kernel.
constexpr int64_t kDequantGemmMinT = 192;
bool gemm_bf16_supported(int64_t T, int64_t K, int64_t ldx, int64_t ldw);
// split_ws (optional, gemm_bf16_split_ws_bytes(T, K, M) bytes, 16-byte
// aligned): lets a projection with too few 128 x 256 tiles run as two K
// slices plus an ordered sum (only without the low-rank epilogue).
hipError_t launch_gemm_bf16(const uint16_t* X, int64_t T, int64_t K, int64_t ldx, const uint16_t* Wq,
                            int64_t ldw, int64_t M, void* Y, bool yf32, int64_t ldy, hipStream_t st,
                            StageTimer tm = {}, const LowrankEpilogue* lr = nullptr, float* split_ws = nullptr);
int gemm_bf16_splits(int64_t T, int64_t K, int64_t M);
size_t gemm_bf16_split_ws_bytes(int64_t T, int64_t K, int64_t M);
// Workspace of the prompt-sized projection: the dequantized weight (M x K
// bf16), then, 256-byte aligned, the K-slice partials.
inline size_t dequant_ws_bytes(int64_t M, int64_t K) {
    return ((size_t)M * (size_t)K * 2 + 255) / 256 * 256;
}
inline float* split_ws_after(uint16_t* wq, int64_t M, int64_t K) {
    return wq ? (float*)((char*)wq + dequant_ws_bytes(M, K)) : nullptr;
}
// Few-token projection (decode steps and short prompts): T <= kQgemvMaxT,
// K a multiple of 128 (at most 16384 for T > 4).  A batch of P prompts
// (T <= 4 only) reads prompt p's operands at the element strides of bt.
constexpr int64_t kQgemvMaxT = 128;
constexpr int64_t kQgemvBatchMaxT = 4;
struct QgemvBatch {
    int64_t x = 0, s = 0, codes = 0, sz = 0, y = 0;
};
bool qgemv_supported(int64_t T, int64_t K, int64_t ldx, bool xf32);
// kGsMinT <= T <= 16, bf16 X, 4-bit codes, groups of 32/64/128, K a
// multiple of 128: the group scale applied to sums on the matrix cores
// (qgemv_gs.hip); x/s and its 32-channel sums are formed in LDS by the same
// launch.  A workspace of qgemv_gs_ws_bytes(T, K, M) bytes (256-byte
// aligned; zero when K is not split) holds the fp32 partials of K slices.
constexpr int64_t kGsMinT = 5;
bool qgemv_gs_eligible(int64_t T, int64_t K, int64_t M, int bits, int group, bool xf32, int64_t ldx);
size_t qgemv_gs_ws_bytes(int64_t T, int64_t K, int64_t M);
hipError_t launch_qgemv_gs(const void* X, bool xf32, int64_t T, int64_t K, int64_t ldx, const float* s,
                           const uint32_t* codes, const uint16_t* scale, const uint16_t* zero, int64_t M, int bits,
                           int group, void* Y, bool yf32, int64_t ldy, void* ws, hipStream_t st,
                           StageTimer tm = {}, bool partials = false);
// K slices of the sums path.  With `partials` and several of them, the call
// leaves their fp32 partials [slices][T][M] in ws and Y unwritten.
int qgemv_gs_slices(int64_t T, int64_t K, int64_t M);
// kSkMinT <= T <= 16, bf16 X, K a multiple of 128: split-K variant with an
// fp32 partial workspace P of qgemv_sk_ws_bytes(T, K, M) bytes.
constexpr int64_t kSkMinT = 12;
bool qgemv_sk_eligible(int64_t T, int64_t K, int64_t ldx, bool xf32);
size_t qgemv_sk_ws_bytes(int64_t T, int64_t K, int64_t M);
hipError_t launch_qgemv_sk(const void* X, bool xf32, int64_t T, int64_t K, int64_t ldx, const float* s,
                           const uint32_t* codes, const uint16_t* scale, const uint16_t* zero, int64_t M, int bits,
                           int group, void* Y, bool yf32, int64_t ldy, float* P, hipStream_t st, StageTimer tm = {});
hipError_t launch_qgemv(const void* X, bool xf32, int64_t T, int64_t K, int64_t ldx, const float* s,
                        const uint32_t* codes, const uint16_t* scale, const uint16_t* zero, int64_t M, int bits,
                        int group, void* Y, bool yf32, int64_t ldy, hipStream_t st, StageTimer tm = {},
                        int64_t P = 1, QgemvBatch bt = {});
// Z = X A^T (fp32, [T][rank]) on the matrix cores, for bf16 X, K % 32 == 0
// and a 16-byte-aligned A.
bool lowrank_z_mfma_ok(bool xf32, int64_t T, int64_t K, int64_t ldx, const float* A);
// parts > 1: K is cut into `parts` slices and Z holds their partials
// [parts][T][rank] (lowrank_zm_parts(T, K) fills the chip).
hipError_t launch_lowrank_z(const void* X, bool xf32, int64_t T, int64_t K, int64_t ldx, const float* A,
                            int rank, float* Z, hipStream_t st, StageTimer tm = {}, int parts = 1);
int lowrank_zm_parts(int64_t T, int64_t K);
hipError_t launch_lowrank(const void* X, bool xf32, int64_t T, int64_t K, int64_t ldx,
                          const float* A, const float* B, int64_t M, int rank, void* Y, bool yf32,
                          int64_t ldy, float* Zp, hipStream_t st, StageTimer tm = {});


// Per-prompt low-rank factors (factors.hip): workspace regions and the call.
struct FactorsLayout {
    size_t wt, yp, ym, yk, gp, rinv, g, tb, ta, total;
};
FactorsLayout factors_layout(int64_t M, int64_t K, int l);
bool factors_supported(bool wf32, int64_t M, int64_t K, int64_t ldw, int l, int rank);
hipError_t launch_factors(const uint16_t* W, int64_t M, int64_t K, int64_t ldw, const float* s, const float* om,
                          int l, int q, int rank, float* B, float* A, char* ws, hipStream_t st);

// Router (route.hip): E <= kMoeMaxExperts, topk <= min(E, kRouteMaxTopk).
constexpr int kMoeMaxExperts = 1024;
constexpr int kRouteMaxTopk = 32;
hipError_t launch_moe_route(const void* L, bool lf32, int64_t T, int E, int64_t ldl, int topk, int score, int renorm,
                            int32_t* ids, float* w, hipStream_t st);

// Mixture-of-experts layer (moe.hip), T <= kMoeMaxT.
constexpr int64_t kMoeMaxT = 1024;
size_t moe_ws_bytes(int64_t T, int64_t topk, int64_t K, int64_t I, int64_t M, int64_t E);
hipError_t launch_moe(const ttq_moe_args* a, char* ws, hipStream_t st);

// Projection of fp32 X with x / s to 24 bits (moe_mfma.hip): its partial sums
// [parts][T][M], to be added in order, at the start of ws.
int proj_f32_parts(int64_t T, int64_t K, int64_t M);
size_t proj_f32_ws_bytes(int64_t T, int64_t K, int64_t M);
hipError_t launch_proj_f32(const float* X, int64_t T, int64_t K, int64_t ldx, const float* s, const uint32_t* codes,
                           const uint16_t* scale, const uint16_t* zero, int64_t M, int bits, int group, char* ws,
                           hipStream_t st);

// Adapters of many requests (adapters.hip).
struct AdapterTable {
    const void* A;
    const void* B;
    bool f32;                   // dtype of A and B
    int n, rank;
    const int32_t* ranks;
    const float* scale;
    const int32_t* ids;
};
size_t adapters_ws_bytes(int64_t T, int64_t K, int rank);
// What the adapters are added to: C [T][M] (nullptr: zeros), or `parts` fp32
// partial sums of it, `stride` floats apart.
struct ProjectionIn {
    const void* C;
    bool f32;
    int64_t ldc;
    int parts = 1;
    int64_t stride = 0;
};
hipError_t launch_adapters(const void* X, bool xf32, int64_t T, int64_t K, int64_t ldx, const AdapterTable& ad,
                           const ProjectionIn& c, int64_t M, void* Y, bool yf32, int64_t ldy, float* Z,
                           hipStream_t st);

// Rows in 8 bits (rows_i8.hip): codes [R][K] with row stride ldc, scale [R].
struct I8RowsArgs {
    const void* X;
    bool xf32;
    int64_t ldx;
    int64_t R, K;
    const float* s;             // nullptr: v = x
    bool divide;                // v = x / s, else x s
    int8_t* codes;
    int64_t ldc;
    float* scale;
    // Rows sorted by expert: at most R, *nrows of them; row r is that of X of
    // slot order[r] (token order[r] / topk), with s + ids[slot] * s_stride
    // (ids nullptr: one s).
    const int32_t* nrows = nullptr;
    const int32_t* order = nullptr;
    int topk = 1;
    const int32_t* ids = nullptr;
    int64_t s_stride = 0;
};
hipError_t launch_quantize_rows(const I8RowsArgs& a, hipStream_t st);

// Products of 8-bit codes (gemm_i8.hip).
struct I8Product {
    const int8_t* X;
    int64_t ldx;
    const float* x_scale;
    int64_t T, K;
    const int8_t* W;            // [M][K], with s_down [2 M][K]
    int64_t ldw;
    const float* w_scale;
    int64_t M;
    void* Y;
    int64_t ldy;
    // Rows sorted by expert: row r of Y is the product of row order[r] / topk of
    // X (order nullptr: row r) and, for offsets[e] <= r < offsets[e + 1], of
    // matrix e, w_stride codes behind the one before; T is at least offsets[E].
    const int32_t* offsets = nullptr;
    const int32_t* order = nullptr;
    int topk = 1, E = 1;
    int64_t xrows = 0;          // of X, with order
    int64_t w_stride = 0;
    // Gate and up: Y (fp32) is act(g) u / s_down[e * s_stride + o].
    const float* s_down = nullptr;
    int64_t s_stride = 0;
    int act = 0;
    // Set by the launch:
    int yvec = 0;
    int splits = 1;             // parts of the channels, their sums in `sums`
    int* sums = nullptr;
};
size_t i8_product_ws_bytes(int64_t T, int64_t K, int64_t M);
bool i8_product_fits(int64_t T, int64_t M, int64_t E);   // a grid can cover T x M, for E matrices (0: one, without offsets)
hipError_t launch_i8_product(const I8Product& p, bool yf32, void* ws, hipStream_t st);

// ttq_qgemm_i8 of one token in one launch (codes and scales of X unused).
bool i8_one_fits(int64_t T, int64_t K);
hipError_t launch_i8_one(const I8RowsArgs& x, const I8Product& p, bool yf32, hipStream_t st);

// Tokens sorted by expert and back (sort.hip).
size_t moe_sort_ws_bytes(int64_t n, int64_t E);
hipError_t launch_moe_sort(const int32_t* ids, int64_t n, int E, int32_t* offsets, int32_t* order, int32_t* pos,
                           int32_t* ws, hipStream_t st);
hipError_t launch_moe_gather(const void* X, int es, int64_t T, int64_t K, int64_t ldx, const int32_t* pos, int topk,
                             void* R, int64_t rows, int64_t ldr, hipStream_t st);
hipError_t launch_moe_combine(const void* R, bool rf32, int64_t rows, int64_t ldr, const int32_t* pos, const float* w,
                              int64_t T, int topk, int64_t M, void* Y, bool yf32, int64_t ldy, hipStream_t st);
hipError_t launch_moe_combine_grad(const void* dY, bool yf32, int64_t lddy, const void* R, bool rf32, int64_t rows,
                                   int64_t ldr, const int32_t* pos, const float* w, int64_t T, int topk, int64_t M,
                                   void* dR, int64_t lddr, float* dw, hipStream_t st);

// Mixture-of-experts layer in 8-bit integers (moe_i8.hip).
size_t moe_i8_ws_bytes(int64_t T, int64_t topk, int64_t K, int64_t I, int64_t M, int64_t E);
hipError_t launch_moe_i8(const ttq_moe_i8_args* a, char* ws, hipStream_t st);

// ttq_linear's argument checks (clearing the calling thread's error text
// first) and the workspace bytes the call needs (0 for an empty call).
ttq_status linear_check(const ttq_linear_args* a, size_t* need);
// Record `msg` as the calling thread's last error text; returns st.
ttq_status set_error(ttq_status st, const char* msg);

}  // namespace ttq
