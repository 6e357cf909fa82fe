// The libttq C ABI: argument validation, workspace layout, launches.
//
// Every check runs on the host before any HIP call; a failed check returns
// TTQ_ERR_INVALID / TTQ_ERR_UNSUPPORTED and launches nothing.  Global state:
// the per-thread error text, and a per-device memo of the quantizer's
// residency (a property of the code object, so it never changes a result).
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <string>

#include <hip/hip_runtime.h>

#include "ttq.h"
#include "launch.hpp"

namespace {

thread_local std::string g_last_error;

ttq_status fail(ttq_status st, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
ttq_status fail(ttq_status st, const char* fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    g_last_error = buf;
    return st;
}

ttq_status device_status(hipError_t e, const char* what) {
    if (e == hipSuccess) return TTQ_OK;
    return fail(TTQ_ERR_DEVICE, "%s: %s", what, hipGetErrorString(e));
}

constexpr int64_t kMaxDim = (int64_t)1 << 30;
constexpr int64_t kMaxK = (int64_t)1 << 18;    // input channels (block sums of the mean fit in LDS)
constexpr int kMaxRank = 64;
constexpr size_t kAlign = 256;

bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }
size_t round_up(size_t n) { return (n + kAlign - 1) / kAlign * kAlign; }
bool dtype_ok(int t) { return t == TTQ_F32 || t == TTQ_BF16; }
size_t esize(int t) { return t == TTQ_F32 ? 4 : 2; }
bool bits_ok(int b) { return b >= 2 && b <= 5; }
bool group_ok(int g) { return g == 16 || g == 32 || g == 64 || g == 128; }
bool dim_ok(int64_t n) { return n >= 0 && n <= kMaxDim; }

#define TTQ_REQUIRE(cond, ...)                                \
    do {                                                      \
        if (!(cond)) return fail(TTQ_ERR_INVALID, __VA_ARGS__); \
    } while (0)

// Checks for the output Y [T][M]: element-aligned, any row stride >= M.
ttq_status check_output(const void* p, int t, int64_t rows, int64_t M, int64_t ld) {
    TTQ_REQUIRE(dtype_ok(t), "Y: unknown dtype %d", t);
    TTQ_REQUIRE(ld >= M && ld <= kMaxDim, "Y: row stride %lld < row length %lld", (long long)ld, (long long)M);
    if (rows > 0 && M > 0) {
        TTQ_REQUIRE(p != nullptr, "Y: null pointer");
        TTQ_REQUIRE(aligned(p, esize(t)), "Y: pointer not aligned to its element size");
    }
    return TTQ_OK;
}

// Checks for a [rows][K] row-major matrix argument of dtype t.
ttq_status check_matrix(const char* name, const void* p, int t, int64_t rows, int64_t K, int64_t ld) {
    TTQ_REQUIRE(dtype_ok(t), "%s: unknown dtype %d", name, t);
    TTQ_REQUIRE(ld >= K && ld <= kMaxDim, "%s: row stride %lld < row length %lld", name, (long long)ld, (long long)K);
    if (rows > 0) {
        TTQ_REQUIRE(p != nullptr, "%s: null pointer", name);
        TTQ_REQUIRE(aligned(p, 16), "%s: pointer not 16-byte aligned", name);
        TTQ_REQUIRE((ld * (int64_t)esize(t)) % 16 == 0, "%s: row stride is not a multiple of 16 bytes", name);
    }
    return TTQ_OK;
}

ttq_status check_quant_shape(int64_t M, int64_t K, int bits, int group) {
    TTQ_REQUIRE(dim_ok(M), "M out of range");
    TTQ_REQUIRE(K > 0 && K <= kMaxK && K % 32 == 0, "K must be a positive multiple of 32, at most 2^18");
    if (!bits_ok(bits)) return fail(TTQ_ERR_INVALID, "bits must be 2, 3, 4 or 5 (got %d)", bits);
    if (!group_ok(group)) return fail(TTQ_ERR_INVALID, "group must be 16, 32, 64 or 128 (got %d)", group);
    TTQ_REQUIRE(K % group == 0, "K must be a multiple of the group size");
    return TTQ_OK;
}

ttq_status check_state(const float* s, const void* codes, const void* scale, const void* zero, bool need_s) {
    TTQ_REQUIRE(!need_s || s != nullptr, "s: null pointer");
    TTQ_REQUIRE(s == nullptr || aligned(s, 16), "s: pointer not 16-byte aligned");
    TTQ_REQUIRE(codes != nullptr && aligned(codes, 16), "codes: null or not 16-byte aligned");
    TTQ_REQUIRE(scale != nullptr && aligned(scale, 2), "scale_f16: null or misaligned");
    TTQ_REQUIRE(zero != nullptr && aligned(zero, 2), "zero_f16: null or misaligned");
    return TTQ_OK;
}

ttq_status check_lowrank(const float* B, const float* A, int rank, bool allow_zero) {
    TTQ_REQUIRE(rank >= (allow_zero ? 0 : 1) && rank <= kMaxRank, "rank must be in [%d, %d] (got %d)",
                allow_zero ? 0 : 1, kMaxRank, rank);
    TTQ_REQUIRE((B == nullptr) == (rank == 0) && (A == nullptr) == (rank == 0),
                "B and A must both be given iff rank > 0");
    TTQ_REQUIRE(B == nullptr || (aligned(B, 4) && aligned(A, 4)), "B/A: misaligned");
    return TTQ_OK;
}

ttq_status check_ws(const void* ws, size_t ws_bytes, size_t need) {
    if (need == 0) return TTQ_OK;
    TTQ_REQUIRE(ws != nullptr, "workspace: null pointer (%zu bytes needed)", need);
    TTQ_REQUIRE(aligned(ws, kAlign), "workspace: pointer not 256-byte aligned");
    TTQ_REQUIRE(ws_bytes >= need, "workspace: %zu bytes given, %zu needed", ws_bytes, need);
    return TTQ_OK;
}

// Prompt-sized projections stage the dequantized weight (M x K bf16) in the
// workspace; the size is requested whenever T allows that path.
size_t ws_qgemm(int64_t T, int64_t K, int64_t M) {
    // 5 <= T <= 16: the fp32 partials of the K slices of the sums kernel
    // (4-bit codes) or of the split-K few-token projection.
    if (T >= ttq::kGsMinT && T <= 16 && K % 128 == 0) {
        const size_t gs = round_up(ttq::qgemv_gs_ws_bytes(T, K, M));
        const size_t sk = T >= ttq::kSkMinT ? round_up(ttq::qgemv_sk_ws_bytes(T, K, M)) : 0;
        return gs > sk ? gs : sk;
    }
    if (T < ttq::kDequantGemmMinT) return 0;
    return ttq::dequant_ws_bytes(M, K) + round_up(ttq::gemm_bf16_split_ws_bytes(T, K, M));
}
bool use_dequant_gemm(int64_t T, bool xf32, int64_t K, int64_t ldx) {
    return !xf32 && T >= ttq::kDequantGemmMinT && ttq::gemm_bf16_supported(T, K, ldx, K);
}
size_t ws_lowrank(int64_t T, int64_t K, int rank) {
    if (rank <= 0 || T <= 0) return 0;
    int64_t len = 0;
    int ns = ttq::lowrank_slices(T, K, &len);
    if (ttq::lowrank_zm_parts(T, K) > ns) ns = ttq::lowrank_zm_parts(T, K);
    return round_up((size_t)ns * (size_t)T * (size_t)rank * sizeof(float));
}

struct StateLayout {
    size_t ssq, s, codes, scale, zero, bsum, scratch, total;
};
StateLayout state_layout(int64_t T, int64_t K, int64_t M, int bits, int group, int rank) {
    StateLayout L{};
    size_t off = 0;
    L.ssq = off;     off += round_up((size_t)K * sizeof(double));
    L.s = off;       off += round_up((size_t)K * sizeof(float));
    L.codes = off;   off += round_up((size_t)M * (size_t)(K * bits / 32) * sizeof(int32_t));
    L.scale = off;   off += round_up((size_t)M * (size_t)(K / group) * sizeof(uint16_t));
    L.zero = off;    off += round_up((size_t)M * (size_t)(K / group) * sizeof(uint16_t));
    L.bsum = off;    off += round_up((size_t)((K + 15) / 16) * sizeof(double));
    L.scratch = off;
    size_t scratch = 0;
    // prompt-sized projections: the dequantized weight, then Z = X A^T for
    // the low-rank epilogue
    const size_t proj = ws_qgemm(T, K, M) + (rank > 0 && T > 0 ? round_up((size_t)ttq::lowrank_zm_parts(T, K) *
                                                                          T * rank * sizeof(float)) : 0);
    if (proj > scratch) scratch = proj;
    if (ws_lowrank(T, K, rank) > scratch) scratch = ws_lowrank(T, K, rank);
    L.total = off + scratch;
    return L;
}

hipStream_t as_stream(void* s) { return (hipStream_t)s; }

}  // namespace

extern "C" {

const char* ttq_status_str(int status) {
    switch (status) {
        case TTQ_OK: return "TTQ_OK";
        case TTQ_ERR_INVALID: return "TTQ_ERR_INVALID";
        case TTQ_ERR_UNSUPPORTED: return "TTQ_ERR_UNSUPPORTED";
        case TTQ_ERR_DEVICE: return "TTQ_ERR_DEVICE";
    }
    return "TTQ_ERR_UNKNOWN";
}

const char* ttq_last_error(void) { return g_last_error.c_str(); }

size_t ttq_workspace_bytes(int64_t T, int64_t K, int64_t M, int bits, int group, int rank) {
    if (!dim_ok(T) || !dim_ok(M) || K <= 0 || K > kMaxK || K % 32 || !bits_ok(bits) ||
        !group_ok(group) || K % group || rank < 0 || rank > kMaxRank)
        return 0;
    return state_layout(T, K, M, bits, group, rank).total;
}

ttq_status ttq_stats(const void* X, int xt, int64_t T, int64_t K, int64_t ldx, double* ssq,
                     int accumulate, void* ws, size_t ws_bytes, void* stream) {
    return ttq_stats_p(X, xt, T, K, ldx, 2.0f, ssq, accumulate, ws, ws_bytes, stream);
}

ttq_status ttq_stats_p(const void* X, int xt, int64_t T, int64_t K, int64_t ldx, float p, double* msum,
                       int accumulate, void* ws, size_t ws_bytes, void* stream) {
    g_last_error.clear();
    double* ssq = msum;
    TTQ_REQUIRE(std::isfinite(p) && p > 0.f, "p must be finite and > 0");
    TTQ_REQUIRE(dim_ok(T), "T out of range");
    TTQ_REQUIRE(K > 0 && K <= kMaxK && K % 8 == 0, "K must be a positive multiple of 8, at most 2^18");
    if (ttq_status e = check_matrix("X", X, xt, T, K, ldx)) return e;
    TTQ_REQUIRE(ssq != nullptr && aligned(ssq, 8), "ssq: null or not 8-byte aligned");
    (void)ws;
    (void)ws_bytes;
    if (T == 0 && accumulate) return TTQ_OK;
    return device_status(ttq::launch_stats(X, xt == TTQ_F32, T, K, ldx, ssq, accumulate, as_stream(stream),
                                           nullptr, {}, (double)p),
                         "ttq_stats launch");
}

ttq_status ttq_awq_scales(const double* ssq, int64_t n_tokens, int64_t K, float alpha,
                          float lambda_rel, float p, float* s, void* stream) {
    g_last_error.clear();
    TTQ_REQUIRE(K > 0 && K <= kMaxK, "K must be in [1, 2^18]");
    TTQ_REQUIRE(n_tokens > 0, "n_tokens must be positive");
    TTQ_REQUIRE(ssq != nullptr && aligned(ssq, 8), "ssq: null or not 8-byte aligned");
    TTQ_REQUIRE(s != nullptr && aligned(s, 16), "s: null or not 16-byte aligned");
    TTQ_REQUIRE(std::isfinite(alpha) && alpha >= 0.f, "alpha must be finite and >= 0");
    TTQ_REQUIRE(std::isfinite(lambda_rel) && lambda_rel >= 0.f, "lambda_rel must be finite and >= 0");
    TTQ_REQUIRE(std::isfinite(p) && p > 0.f, "p must be finite and > 0");
    return device_status(ttq::launch_awq_scales(ssq, n_tokens, K, alpha, lambda_rel, p, s, as_stream(stream)),
                         "ttq_awq_scales launch");
}

ttq_status ttq_quantize_groups(const void* W, int wt, int64_t M, int64_t K, int64_t ldw,
                               const float* s, int bits, int group, const float* B, const float* A,
                               int rank, int32_t* codes, uint16_t* scale_f16, uint16_t* zero_f16,
                               void* stream) {
    g_last_error.clear();
    if (ttq_status e = check_quant_shape(M, K, bits, group)) return e;
    if (ttq_status e = check_matrix("W", W, wt, M, K, ldw)) return e;
    if (ttq_status e = check_lowrank(B, A, rank, true)) return e;
    if (M == 0) return TTQ_OK;
    if (ttq_status e = check_state(s, codes, scale_f16, zero_f16, false)) return e;
    return device_status(ttq::launch_quantize(W, wt == TTQ_F32, M, K, ldw, s, bits, group, B, A, rank,
                                              (uint32_t*)codes, scale_f16, zero_f16, nullptr,
                                              as_stream(stream)),
                         "ttq_quantize_groups launch");
}

ttq_status ttq_qgemm(const void* X, int xt, int64_t T, int64_t K, int64_t ldx, const float* s,
                     const int32_t* codes, const uint16_t* scale_f16, const uint16_t* zero_f16,
                     int64_t M, int bits, int group, void* Y, int yt, int64_t ldy, void* ws,
                     size_t ws_bytes, void* stream) {
    g_last_error.clear();
    TTQ_REQUIRE(dim_ok(T), "T out of range");
    if (ttq_status e = check_quant_shape(M, K, bits, group)) return e;
    if (ttq_status e = check_matrix("X", X, xt, T, K, ldx)) return e;
    if (ttq_status e = check_output(Y, yt, T, M, ldy)) return e;
    if (T == 0 || M == 0) return TTQ_OK;
    if (ttq_status e = check_state(s, codes, scale_f16, zero_f16, true)) return e;
    const bool xf32 = xt == TTQ_F32;
    const bool dq = use_dequant_gemm(T, xf32, K, ldx);
    const bool gs = ttq::qgemv_gs_eligible(T, K, M, bits, group, xf32, ldx);
    const bool sk = !gs && ttq::qgemv_sk_eligible(T, K, ldx, xf32);
    if (ttq_status e = check_ws(ws, ws_bytes, (dq || sk || gs) ? ws_qgemm(T, K, M) : 0)) return e;
    hipStream_t st = as_stream(stream);
    if (gs)
        return device_status(ttq::launch_qgemv_gs(X, xf32, T, K, ldx, s, (const uint32_t*)codes, scale_f16, zero_f16,
                                                  M, bits, group, Y, yt == TTQ_F32, ldy, ws, st),
                             "ttq_qgemm launch");
    if (sk)
        return device_status(ttq::launch_qgemv_sk(X, xf32, T, K, ldx, s, (const uint32_t*)codes, scale_f16, zero_f16,
                                                  M, bits, group, Y, yt == TTQ_F32, ldy, (float*)ws, st),
                             "ttq_qgemm launch");
    if (ttq::qgemv_supported(T, K, ldx, xf32))
        return device_status(ttq::launch_qgemv(X, xf32, T, K, ldx, s, (const uint32_t*)codes, scale_f16, zero_f16,
                                               M, bits, group, Y, yt == TTQ_F32, ldy, st),
                             "ttq_qgemm launch");
    return device_status(ttq::launch_qgemm(X, xf32, T, K, ldx, s, (const uint32_t*)codes,
                                           scale_f16, zero_f16, M, bits, group, Y, yt == TTQ_F32, ldy,
                                           dq ? (uint16_t*)ws : nullptr, st),
                         "ttq_qgemm launch");
}

size_t ttq_lowrank_factors_workspace_bytes(int64_t M, int64_t K, int l) {
    if (M <= 0 || K <= 0 || K > kMaxK || !dim_ok(M) || l < 1 || l > 32) return 0;
    return ttq::factors_layout(M, K, l).total;
}

ttq_status ttq_lowrank_factors(const void* W, int wt, int64_t M, int64_t K, int64_t ldw, const float* s,
                               const float* omega, int l, int q, int rank, float* B, float* A, void* ws,
                               size_t ws_bytes, void* stream) {
    g_last_error.clear();
    TTQ_REQUIRE(dim_ok(M) && M > 0, "M must be positive");
    TTQ_REQUIRE(K > 0 && K <= kMaxK && K % 32 == 0, "K must be a positive multiple of 32, at most 2^18");
    if (ttq_status e = check_matrix("W", W, wt, M, K, ldw)) return e;
    TTQ_REQUIRE(l >= 1 && l <= 32, "l (test vectors) must be in [1, 32]");
    TTQ_REQUIRE(rank >= 1 && rank <= l, "rank must be in [1, l]");
    TTQ_REQUIRE(l <= M && l <= K, "l must not exceed M or K");
    TTQ_REQUIRE(q >= 0 && q <= 64, "q (power iterations) must be in [0, 64]");
    TTQ_REQUIRE(s != nullptr && aligned(s, 4), "s: null or misaligned");
    TTQ_REQUIRE(omega != nullptr && aligned(omega, 4), "omega: null or misaligned");
    TTQ_REQUIRE(B != nullptr && aligned(B, 4) && A != nullptr && aligned(A, 4), "B/A: null or misaligned");
    if (wt == TTQ_F32) return fail(TTQ_ERR_UNSUPPORTED, "per-prompt factors need a bf16 weight");
    TTQ_REQUIRE(ttq::factors_supported(false, M, K, ldw, l, rank), "sizes exceed the factor kernels' addressing");
    if (ttq_status e = check_ws(ws, ws_bytes, ttq::factors_layout(M, K, l).total)) return e;
    return device_status(ttq::launch_factors((const uint16_t*)W, M, K, ldw, s, omega, l, q, rank, B, A, (char*)ws,
                                             as_stream(stream)),
                         "ttq_lowrank_factors launch");
}

ttq_status ttq_qgemm_batched(const void* X, int xt, int64_t P, int64_t T, int64_t K, int64_t ldx,
                             int64_t x_stride, const float* s, int64_t s_stride, const int32_t* codes,
                             int64_t codes_stride, const uint16_t* scale_f16, const uint16_t* zero_f16,
                             int64_t sz_stride, int64_t M, int bits, int group, void* Y, int yt, int64_t ldy,
                             int64_t y_stride, void* stream) {
    g_last_error.clear();
    TTQ_REQUIRE(P >= 1 && P <= 65535, "P (prompts) must be in [1, 65535]");
    TTQ_REQUIRE(T >= 1 && T <= ttq::kQgemvBatchMaxT, "T must be in [1, %d] for batched decode steps",
                (int)ttq::kQgemvBatchMaxT);
    if (ttq_status e = check_quant_shape(M, K, bits, group)) return e;
    TTQ_REQUIRE(K % 128 == 0, "K must be a multiple of 128");
    if (ttq_status e = check_matrix("X", X, xt, T, K, ldx)) return e;
    if (ttq_status e = check_output(Y, yt, T, M, ldy)) return e;
    if (M == 0) return TTQ_OK;
    if (ttq_status e = check_state(s, codes, scale_f16, zero_f16, true)) return e;
    const int64_t xe = esize(xt);
    TTQ_REQUIRE(x_stride >= 0 && (x_stride * xe) % 16 == 0 && (P == 1 || x_stride >= (T - 1) * ldx + K),
                "x_stride: negative, not a multiple of 16 bytes, or overlapping prompts");
    TTQ_REQUIRE(s_stride >= 0 && s_stride % 4 == 0, "s_stride: negative or not a multiple of 16 bytes");
    TTQ_REQUIRE(codes_stride >= 0 && codes_stride % 4 == 0, "codes_stride: negative or not a multiple of 16 bytes");
    TTQ_REQUIRE(sz_stride >= 0, "sz_stride: negative");
    TTQ_REQUIRE(y_stride >= 0 && (P == 1 || y_stride >= (T - 1) * ldy + M), "y_stride: negative or overlapping prompts");
    ttq::QgemvBatch bt;
    bt.x = x_stride; bt.s = s_stride; bt.codes = codes_stride; bt.sz = sz_stride; bt.y = y_stride;
    return device_status(ttq::launch_qgemv(X, xt == TTQ_F32, T, K, ldx, s, (const uint32_t*)codes, scale_f16, zero_f16,
                                           M, bits, group, Y, yt == TTQ_F32, ldy, as_stream(stream), {}, P, bt),
                         "ttq_qgemm_batched launch");
}

ttq_status ttq_lowrank_add(const void* X, int xt, int64_t T, int64_t K, int64_t ldx, const float* A,
                           const float* B, int64_t M, int rank, void* Y, int yt, int64_t ldy, void* ws,
                           size_t ws_bytes, void* stream) {
    g_last_error.clear();
    TTQ_REQUIRE(dim_ok(T) && dim_ok(M), "T or M out of range");
    TTQ_REQUIRE(K > 0 && K <= kMaxK && K % 8 == 0, "K must be a positive multiple of 8, at most 2^18");
    if (ttq_status e = check_lowrank(B, A, rank, false)) return e;
    if (ttq_status e = check_matrix("X", X, xt, T, K, ldx)) return e;
    if (ttq_status e = check_output(Y, yt, T, M, ldy)) return e;
    if (T == 0 || M == 0) return TTQ_OK;
    if (ttq_status e = check_ws(ws, ws_bytes, ws_lowrank(T, K, rank))) return e;
    return device_status(ttq::launch_lowrank(X, xt == TTQ_F32, T, K, ldx, A, B, M, rank, Y, yt == TTQ_F32,
                                             ldy, (float*)ws, as_stream(stream)),
                         "ttq_lowrank_add launch");
}

static ttq_status check_linear(const ttq_linear_args* a) {
    TTQ_REQUIRE(a != nullptr, "args: null pointer");
    TTQ_REQUIRE(dim_ok(a->T), "T out of range");
    if (ttq_status e = check_quant_shape(a->M, a->K, a->bits, a->group)) return e;
    if (ttq_status e = check_matrix("X", a->X, a->xt, a->T, a->K, a->ldx)) return e;
    if (ttq_status e = check_matrix("W", a->W, a->wt, a->M, a->K, a->ldw)) return e;
    if (ttq_status e = check_output(a->Y, a->yt, a->T, a->M, a->ldy)) return e;
    if (ttq_status e = check_lowrank(a->B, a->A, a->rank, true)) return e;
    TTQ_REQUIRE(std::isfinite(a->alpha) && a->alpha >= 0.f, "alpha must be finite and >= 0");
    TTQ_REQUIRE(std::isfinite(a->lambda_rel) && a->lambda_rel >= 0.f, "lambda_rel must be finite and >= 0");
    TTQ_REQUIRE(std::isfinite(a->p) && a->p > 0.f, "p must be finite and > 0");
    TTQ_REQUIRE(a->ssq == nullptr || aligned(a->ssq, 8), "ssq: not 8-byte aligned");
    TTQ_REQUIRE(a->s == nullptr || aligned(a->s, 16), "s: not 16-byte aligned");
    TTQ_REQUIRE(a->codes == nullptr || aligned(a->codes, 16), "codes: not 16-byte aligned");
    TTQ_REQUIRE(a->scale_f16 == nullptr || aligned(a->scale_f16, 2), "scale_f16: misaligned");
    TTQ_REQUIRE(a->zero_f16 == nullptr || aligned(a->zero_f16, 2), "zero_f16: misaligned");
    if (a->stage_events != nullptr)
        for (int i = 0; i < TTQ_LINEAR_STAGE_EVENTS; ++i)
            TTQ_REQUIRE(a->stage_events[i] != nullptr, "stage_events[%d]: null handle", i);
    return TTQ_OK;
}

// Stage i of ttq_linear is timed by events (2i, 2i+1), stamped by the
// stage's first and last kernel; a stage that launches nothing records both
// on the stream as markers.
struct StageMarks {
    void* const* ev;
    hipStream_t st;
    ttq::StageTimer timer(int i) const {
        if (ev == nullptr) return {};
        return {(hipEvent_t)ev[2 * i], (hipEvent_t)ev[2 * i + 1]};
    }
    ttq_status markers(int i) const {
        if (ev == nullptr) return TTQ_OK;
        for (int k = 0; k < 2; ++k)
            if (ttq_status e = device_status(hipEventRecord((hipEvent_t)ev[2 * i + k], st), "stage event"))
                return e;
        return TTQ_OK;
    }
};

// Everything after the statistics (ssq, and the block sums of c in bsum):
// scales, quantizer, projection and low-rank term, with the state and
// scratch regions of L in w.
static ttq_status linear_layer(const ttq_linear_args* a, const double* ssq, const double* bsum, char* w,
                               const StateLayout& L, hipStream_t st) {
    float* s = a->s ? a->s : (float*)(w + L.s);
    int32_t* codes = a->codes ? a->codes : (int32_t*)(w + L.codes);
    uint16_t* scale = a->scale_f16 ? a->scale_f16 : (uint16_t*)(w + L.scale);
    uint16_t* zero = a->zero_f16 ? a->zero_f16 : (uint16_t*)(w + L.zero);
    void* scratch = w + L.scratch;
    const bool xf32 = a->xt == TTQ_F32;
    const StageMarks sm{a->stage_events, st};
    auto timer = [&](int i) { return sm.timer(i); };
    auto markers = [&](int i) { return sm.markers(i); };
    if (a->M == 0) {
        // No rows to quantize: the scales still form part of the prompt state.
        if (ttq_status e = device_status(ttq::launch_awq_scales(ssq, a->T, a->K, a->alpha, a->lambda_rel, a->p, s, st),
                                         "scales"))
            return e;
        for (int i = 1; i < 4; ++i)
            if (ttq_status e = markers(i)) return e;
        return TTQ_OK;
    }
    // The quantizer evaluates the scales of its channels from (ssq, lambda)
    // with the same arithmetic as ttq_awq_scales, and stores s.
    const ttq::QScaleSrc qs{ssq, bsum, (double)a->lambda_rel, (double)a->T, (double)a->alpha / (double)a->p, s};
    // Prompt-sized projections: the quantizer also writes the dequantized
    // weight (into the scratch area, free again once the statistics are
    // reduced) and the projection is a plain matrix-core GEMM on it.
    const bool dq = use_dequant_gemm(a->T, xf32, a->K, a->ldx);
    uint16_t* wq = dq ? (uint16_t*)scratch : nullptr;
    if (ttq_status e = device_status(
            ttq::launch_quantize(a->W, a->wt == TTQ_F32, a->M, a->K, a->ldw, s, a->bits, a->group, a->B,
                                 a->A, a->rank, (uint32_t*)codes, scale, zero, wq, st, &qs, timer(1)),
            "quantize"))
        return e;
    if (ttq::qgemv_gs_eligible(a->T, a->K, a->M, a->bits, a->group, xf32, a->ldx)) {
        if (ttq_status e = device_status(
                ttq::launch_qgemv_gs(a->X, xf32, a->T, a->K, a->ldx, s, (const uint32_t*)codes, scale, zero, a->M,
                                     a->bits, a->group, a->Y, a->yt == TTQ_F32, a->ldy, scratch, st, timer(2)),
                "qgemv"))
            return e;
    } else if (ttq::qgemv_sk_eligible(a->T, a->K, a->ldx, xf32)) {
        if (ttq_status e = device_status(
                ttq::launch_qgemv_sk(a->X, xf32, a->T, a->K, a->ldx, s, (const uint32_t*)codes, scale, zero, a->M,
                                     a->bits, a->group, a->Y, a->yt == TTQ_F32, a->ldy, (float*)scratch, st,
                                     timer(2)),
                "qgemv"))
            return e;
    } else if (ttq::qgemv_supported(a->T, a->K, a->ldx, xf32)) {
        if (ttq_status e = device_status(
                ttq::launch_qgemv(a->X, xf32, a->T, a->K, a->ldx, s, (const uint32_t*)codes, scale, zero, a->M,
                                  a->bits, a->group, a->Y, a->yt == TTQ_F32, a->ldy, st, timer(2)),
                "qgemv"))
            return e;
    } else if (dq) {
        // With low-rank factors: Z = X A^T on the matrix cores first, then the
        // GEMM adds Z B^T in its epilogue (no second pass over Y).
        ttq::LowrankEpilogue lre{nullptr, a->B, a->rank};
        const bool fuse = a->rank > 0 && ttq::lowrank_z_mfma_ok(xf32, a->T, a->K, a->ldx, a->A);
        if (fuse) {
            float* Z = (float*)((char*)scratch + ws_qgemm(a->T, a->K, a->M));
            lre.nz = ttq::lowrank_zm_parts(a->T, a->K);
            if (ttq_status e = device_status(ttq::launch_lowrank_z(a->X, xf32, a->T, a->K, a->ldx, a->A, a->rank, Z,
                                                                   st, timer(3), lre.nz),
                                             "lowrank Z"))
                return e;
            lre.Z = Z;
        }
        if (ttq_status e = device_status(ttq::launch_gemm_bf16((const uint16_t*)a->X, a->T, a->K, a->ldx, wq,
                                                               a->K, a->M, a->Y, a->yt == TTQ_F32, a->ldy, st,
                                                               timer(2), fuse ? &lre : nullptr,
                                                               fuse ? nullptr : ttq::split_ws_after(wq, a->M, a->K)),
                                         "gemm"))
            return e;
        if (fuse) return TTQ_OK;
    } else if (ttq_status e = device_status(
                   ttq::launch_qgemm(a->X, xf32, a->T, a->K, a->ldx, s, (const uint32_t*)codes, scale, zero,
                                     a->M, a->bits, a->group, a->Y, a->yt == TTQ_F32, a->ldy, nullptr, st,
                                     timer(2)),
                   "qgemm")) {
        return e;
    }
    if (a->rank > 0)
        return device_status(ttq::launch_lowrank(a->X, xf32, a->T, a->K, a->ldx, a->A, a->B, a->M, a->rank, a->Y,
                                                 a->yt == TTQ_F32, a->ldy, (float*)scratch, st, timer(3)),
                             "lowrank");
    return markers(3);
}

}  // extern "C"

namespace ttq {

ttq_status linear_check(const ttq_linear_args* a, size_t* need) {
    g_last_error.clear();
    if (ttq_status e = check_linear(a)) return e;
    *need = a->T == 0 ? 0 : state_layout(a->T, a->K, a->M, a->bits, a->group, a->rank).total;
    return TTQ_OK;
}

ttq_status set_error(ttq_status st, const char* msg) { return fail(st, "%s", msg); }

}  // namespace ttq

extern "C" {

ttq_status ttq_linear(const ttq_linear_args* a, void* ws, size_t ws_bytes, void* stream) {
    g_last_error.clear();
    if (ttq_status e = check_linear(a)) return e;
    if (a->T == 0) return TTQ_OK;   // no prompt tokens: nothing to estimate or project
    const StateLayout L = state_layout(a->T, a->K, a->M, a->bits, a->group, a->rank);
    if (ttq_status e = check_ws(ws, ws_bytes, L.total)) return e;
    char* w = (char*)ws;
    double* ssq = a->ssq ? a->ssq : (double*)(w + L.ssq);
    double* bsum = (double*)(w + L.bsum);
    hipStream_t st = as_stream(stream);
    // Statistics (sums of |x|^p); the reduction also leaves the 16-channel
    // block sums of c.
    const StageMarks sm{a->stage_events, st};
    if (ttq_status e = device_status(ttq::launch_stats(a->X, a->xt == TTQ_F32, a->T, a->K, a->ldx, ssq, 0, st,
                                                       bsum, sm.timer(0), (double)a->p),
                                     "stats"))
        return e;
    return linear_layer(a, ssq, bsum, w, L, st);
}

// Shared statistics: [ssq K fp64 | block sums] at the head of the workspace,
// then one layer's state and scratch at a time (layers run in order).
static size_t shared_head(int64_t K) { return round_up((size_t)K * 8) + round_up((size_t)((K + 15) / 16) * 8); }

size_t ttq_linear_shared_workspace_bytes(const ttq_linear_args* layers, int n) {
    if (layers == nullptr || n < 1) return 0;
    size_t mx = 0;
    for (int i = 0; i < n; ++i) {
        const ttq_linear_args* a = &layers[i];
        if (ttq_workspace_bytes(a->T, a->K, a->M, a->bits, a->group, a->rank) == 0) return 0;
        const size_t t = state_layout(a->T, a->K, a->M, a->bits, a->group, a->rank).total;
        if (t > mx) mx = t;
    }
    return shared_head(layers[0].K) + mx;
}

ttq_status ttq_linear_shared(const ttq_linear_args* layers, int n, void* ws, size_t ws_bytes, void* stream) {
    g_last_error.clear();
    TTQ_REQUIRE(layers != nullptr && n >= 1 && n <= 64, "layers: null, or n not in [1, 64]");
    const ttq_linear_args* a0 = &layers[0];
    for (int i = 0; i < n; ++i) {
        const ttq_linear_args* a = &layers[i];
        if (ttq_status e = check_linear(a)) return e;
        TTQ_REQUIRE(a->X == a0->X && a->xt == a0->xt && a->T == a0->T && a->K == a0->K && a->ldx == a0->ldx,
                    "layer %d: X, xt, T, K and ldx must equal layer 0's (one shared input)", i);
        TTQ_REQUIRE(a->alpha == a0->alpha && a->lambda_rel == a0->lambda_rel && a->p == a0->p,
                    "layer %d: alpha, lambda_rel and p must equal layer 0's", i);
        TTQ_REQUIRE(a->stage_events == nullptr, "layer %d: stage events are not recorded for shared layers", i);
        TTQ_REQUIRE(i == 0 || a->ssq == nullptr, "layer %d: only layer 0 receives the shared statistics", i);
    }
    if (a0->T == 0) return TTQ_OK;
    const size_t need = ttq_linear_shared_workspace_bytes(layers, n);
    TTQ_REQUIRE(need > 0, "sizes not accepted");
    if (ttq_status e = check_ws(ws, ws_bytes, need)) return e;
    char* w = (char*)ws;
    const size_t head = shared_head(a0->K);
    double* ssq = a0->ssq ? a0->ssq : (double*)w;
    double* bsum = (double*)(w + round_up((size_t)a0->K * 8));
    char* wl = w + head;
    hipStream_t st = as_stream(stream);
    if (ttq_status e = device_status(ttq::launch_stats(a0->X, a0->xt == TTQ_F32, a0->T, a0->K, a0->ldx, ssq, 0, st,
                                                       bsum, {}, (double)a0->p),
                                     "stats"))
        return e;
    for (int i = 0; i < n; ++i) {
        const ttq_linear_args* a = &layers[i];
        const StateLayout L = state_layout(a->T, a->K, a->M, a->bits, a->group, a->rank);
        if (ttq_status e = linear_layer(a, ssq, bsum, wl, L, st)) return e;
    }
    return TTQ_OK;
}

}  // extern "C"

// ------------------------------------------------- weights chosen per token

namespace {

constexpr int64_t kMaxAdapters = 65536;
constexpr int64_t kMaxExpertBytes = (int64_t)1 << 31;   // of one weight's codes: one buffer descriptor
constexpr int64_t kMaxAdapterLdx = (int64_t)1 << 24;

ttq_status check_experts(const char* name, const ttq_expert_state& q, int64_t K) {
    TTQ_REQUIRE(q.s != nullptr && aligned(q.s, 16), "%s.s: null or not 16-byte aligned", name);
    TTQ_REQUIRE(q.s_stride == 0 || (q.s_stride >= K && q.s_stride % 4 == 0 && q.s_stride <= kMaxDim),
                "%s.s_stride: neither 0 nor a multiple of 4 of at least the row length", name);
    return check_state(q.s, q.codes, q.scale_f16, q.zero_f16, true);
}

ttq_status check_moe_sizes(int64_t T, int64_t topk, int64_t K, int64_t I, int64_t M, int64_t E, int bits, int group) {
    TTQ_REQUIRE(dim_ok(T), "T out of range");
    TTQ_REQUIRE(E >= 1 && E <= ttq::kMoeMaxExperts, "E (experts) must be in [1, %d]", ttq::kMoeMaxExperts);
    TTQ_REQUIRE(topk >= 1 && topk <= ttq::kRouteMaxTopk, "topk must be in [1, %d]", ttq::kRouteMaxTopk);
    if (ttq_status e = check_quant_shape(M, K, bits, group)) return e;
    TTQ_REQUIRE(I > 0 && I <= kMaxK && I % 32 == 0 && I % group == 0,
                "I must be a positive multiple of 32 and of the group size, at most 2^18");
    if (2 * I * K * bits / 8 >= kMaxExpertBytes || M * I * bits / 8 >= kMaxExpertBytes)
        return fail(TTQ_ERR_UNSUPPORTED, "an expert's codes take 2 GiB or more");
    if (T > ttq::kMoeMaxT)
        return fail(TTQ_ERR_UNSUPPORTED, "at most %d tokens a call (got %lld): pass a longer prompt in chunks",
                    (int)ttq::kMoeMaxT, (long long)T);
    return TTQ_OK;
}

// X, C and Y are checked by the caller.
ttq_status check_adapters(const ttq_adapters* ad, int64_t T, int64_t K, int64_t ldx) {
    TTQ_REQUIRE(ad != nullptr, "adapters: null pointer");
    TTQ_REQUIRE(dtype_ok(ad->dt), "adapters: unknown dtype %d", ad->dt);
    TTQ_REQUIRE(ad->n >= 0 && ad->n <= kMaxAdapters, "adapters: n must be in [0, %d]", (int)kMaxAdapters);
    TTQ_REQUIRE(ad->rank >= 1 && ad->rank <= kMaxRank, "adapters: rank must be in [1, %d] (got %d)", kMaxRank, ad->rank);
    TTQ_REQUIRE(K > 0 && K <= kMaxK && K % 8 == 0, "K must be a positive multiple of 8, at most 2^18");
    TTQ_REQUIRE(ad->n == 0 || (ad->A != nullptr && aligned(ad->A, 16) && ad->B != nullptr && aligned(ad->B, 16)),
                "adapters: A or B null or not 16-byte aligned");
    TTQ_REQUIRE(aligned(ad->ranks, 4) && aligned(ad->scale, 4), "adapters: ranks or scale misaligned");
    TTQ_REQUIRE(T == 0 || (ad->ids != nullptr && aligned(ad->ids, 4)), "adapters: ids null or misaligned");
    if (ldx > kMaxAdapterLdx)   // 16 rows lie within one buffer descriptor
        return fail(TTQ_ERR_UNSUPPORTED, "X: row stride above 2^24 elements");
    return TTQ_OK;
}

ttq::AdapterTable adapter_table(const ttq_adapters* ad) {
    return {ad->A, ad->B, ad->dt == TTQ_F32, (int)ad->n, ad->rank, ad->ranks, ad->scale, ad->ids};
}

// fp32 X: four tokens at most have a projection in fp32 arithmetic
// (launch_qgemv); ttq_qgemm's other ones keep 16 bits of x / s, this one 24.
bool shared_f32(int64_t T, int64_t K) { return T > 4 || K % 128 != 0; }

// Workspace of ttq_qgemm_adapters: the adapters' sums, then the projection in
// fp32 and its own workspace, or that of the projection of fp32 X.
struct SharedLayout {
    size_t z, c, q, total;
};
SharedLayout shared_layout(int64_t T, int64_t K, int64_t M, int rank) {
    SharedLayout L{};
    L.z = 0;
    L.c = L.z + round_up(ttq::adapters_ws_bytes(T, K, rank));
    L.q = L.c + round_up((size_t)T * (size_t)M * 4);
    L.total = L.q + ws_qgemm(T, K, M);
    const size_t f32 = L.c + (shared_f32(T, K) ? ttq::proj_f32_ws_bytes(T, K, M) : 0);
    if (L.total < f32) L.total = f32;
    return L;
}

}  // namespace

extern "C" {

ttq_status ttq_moe_route(const void* logits, int lt, int64_t T, int64_t E, int64_t ldl, int topk, int score,
                         int renormalize, int32_t* ids, float* w, void* stream) {
    g_last_error.clear();
    TTQ_REQUIRE(dim_ok(T), "T out of range");
    TTQ_REQUIRE(E >= 1 && E <= ttq::kMoeMaxExperts, "E (experts) must be in [1, %d]", ttq::kMoeMaxExperts);
    TTQ_REQUIRE(topk >= 1 && topk <= E && topk <= ttq::kRouteMaxTopk, "topk must be in [1, min(E, %d)]",
                ttq::kRouteMaxTopk);
    TTQ_REQUIRE(dtype_ok(lt), "logits: unknown dtype %d", lt);
    TTQ_REQUIRE(ldl >= E && ldl <= kMaxDim, "logits: row stride %lld < E", (long long)ldl);
    TTQ_REQUIRE(score == TTQ_SCORE_SOFTMAX || score == TTQ_SCORE_SIGMOID, "score: unknown value %d", score);
    if (T == 0) return TTQ_OK;
    TTQ_REQUIRE(logits != nullptr && aligned(logits, esize(lt)), "logits: null or misaligned");
    TTQ_REQUIRE(ids != nullptr && aligned(ids, 4) && w != nullptr && aligned(w, 4), "ids or w: null or misaligned");
    return device_status(ttq::launch_moe_route(logits, lt == TTQ_F32, T, (int)E, ldl, topk, score, renormalize != 0,
                                               ids, w, as_stream(stream)),
                         "ttq_moe_route launch");
}

size_t ttq_moe_workspace_bytes(int64_t T, int64_t topk, int64_t K, int64_t I, int64_t M, int64_t E, int bits,
                               int group) {
    if (check_moe_sizes(T, topk, K, I, M, E, bits, group)) return 0;
    return ttq::moe_ws_bytes(T, topk, K, I, M, E) + kAlign;
}

ttq_status ttq_moe(const ttq_moe_args* a, void* ws, size_t ws_bytes, void* stream) {
    g_last_error.clear();
    TTQ_REQUIRE(a != nullptr, "args: null pointer");
    if (ttq_status e = check_moe_sizes(a->T, a->topk, a->K, a->I, a->M, a->E, a->bits, a->group)) return e;
    TTQ_REQUIRE(a->act == TTQ_ACT_SILU || a->act == TTQ_ACT_GELU_TANH, "act: unknown value %d", a->act);
    if (ttq_status e = check_matrix("X", a->X, a->xt, a->T, a->K, a->ldx)) return e;
    if (ttq_status e = check_output(a->Y, a->yt, a->T, a->M, a->ldy)) return e;
    if (a->T == 0 || a->M == 0) return TTQ_OK;
    TTQ_REQUIRE(a->ids != nullptr && aligned(a->ids, 4) && a->w != nullptr && aligned(a->w, 4),
                "ids or w: null or misaligned");
    if (ttq_status e = check_experts("gate_up", a->gate_up, a->K)) return e;
    if (ttq_status e = check_experts("down", a->down, a->I)) return e;
    if (ttq_status e = check_ws(ws, ws_bytes, ttq::moe_ws_bytes(a->T, a->topk, a->K, a->I, a->M, a->E))) return e;
    return device_status(ttq::launch_moe(a, (char*)ws, as_stream(stream)), "ttq_moe launch");
}

size_t ttq_adapters_workspace_bytes(int64_t T, int64_t K, int64_t M, int rank) {
    if (!dim_ok(T) || !dim_ok(M) || K <= 0 || K > kMaxK || K % 8 || rank < 1 || rank > kMaxRank) return 0;
    return round_up(ttq::adapters_ws_bytes(T, K, rank)) + kAlign;
}

ttq_status ttq_adapters_add(const void* X, int xt, int64_t T, int64_t K, int64_t ldx, const ttq_adapters* ad,
                            int64_t M, const void* C, int64_t ldc, void* Y, int yt, int64_t ldy, void* ws,
                            size_t ws_bytes, void* stream) {
    g_last_error.clear();
    TTQ_REQUIRE(dim_ok(T) && dim_ok(M), "T or M out of range");
    if (ttq_status e = check_adapters(ad, T, K, ldx)) return e;
    if (ttq_status e = check_matrix("X", X, xt, T, K, ldx)) return e;
    if (ttq_status e = check_output(Y, yt, T, M, ldy)) return e;
    if (C != nullptr) {
        TTQ_REQUIRE(aligned(C, esize(yt)), "C: pointer not aligned to its element size");
        TTQ_REQUIRE(ldc >= M && ldc <= kMaxDim, "C: row stride %lld < row length %lld", (long long)ldc, (long long)M);
        TTQ_REQUIRE(C != Y || ldc == ldy, "C: in place with another row stride than Y");
    }
    if (T == 0 || M == 0) return TTQ_OK;
    if (ttq_status e = check_ws(ws, ws_bytes, ttq_adapters_workspace_bytes(T, K, M, ad->rank))) return e;
    return device_status(ttq::launch_adapters(X, xt == TTQ_F32, T, K, ldx, adapter_table(ad), {C, yt == TTQ_F32, ldc},
                                              M, Y, yt == TTQ_F32, ldy, (float*)ws, as_stream(stream)),
                         "ttq_adapters_add launch");
}

size_t ttq_qgemm_adapters_workspace_bytes(int64_t T, int64_t K, int64_t M, int bits, int group, int rank) {
    if (!dim_ok(T) || !dim_ok(M) || K <= 0 || K > kMaxK || K % 32 || !bits_ok(bits) || !group_ok(group) ||
        K % group || rank < 1 || rank > kMaxRank)
        return 0;
    return shared_layout(T, K, M, rank).total + kAlign;
}

ttq_status ttq_qgemm_adapters(const void* X, int xt, int64_t T, int64_t K, int64_t ldx, const float* s,
                              const int32_t* codes, const uint16_t* scale_f16, const uint16_t* zero_f16, int64_t M,
                              int bits, int group, const ttq_adapters* ad, void* Y, int yt, int64_t ldy, void* ws,
                              size_t ws_bytes, void* stream) {
    g_last_error.clear();
    TTQ_REQUIRE(dim_ok(T), "T out of range");
    if (ttq_status e = check_quant_shape(M, K, bits, group)) return e;
    if (ttq_status e = check_adapters(ad, T, K, ldx)) return e;
    if (ttq_status e = check_matrix("X", X, xt, T, K, ldx)) return e;
    if (ttq_status e = check_output(Y, yt, T, M, ldy)) return e;
    if (T == 0 || M == 0) return TTQ_OK;
    if (ttq_status e = check_state(s, codes, scale_f16, zero_f16, true)) return e;
    const SharedLayout L = shared_layout(T, K, M, ad->rank);
    if (ttq_status e = check_ws(ws, ws_bytes, L.total)) return e;
    char* w = (char*)ws;
    float* C = (float*)(w + L.c);
    const bool xf32 = xt == TTQ_F32;
    ttq::ProjectionIn ci{C, true, M};
    if (xf32 && shared_f32(T, K)) {
        if (ttq_status e = device_status(
                ttq::launch_proj_f32((const float*)X, T, K, ldx, s, (const uint32_t*)codes, scale_f16, zero_f16, M, bits,
                                     group, w + L.c, as_stream(stream)),
                "ttq_qgemm_adapters launch"))
            return e;
        ci.parts = ttq::proj_f32_parts(T, K, M);
        ci.stride = T * M;
    } else if (ttq::qgemv_gs_eligible(T, K, M, bits, group, xf32, ldx)) {
        // The K slices' partial sums are added where the adapters are.
        if (ttq_status e = device_status(
                ttq::launch_qgemv_gs(X, xf32, T, K, ldx, s, (const uint32_t*)codes, scale_f16, zero_f16, M, bits, group,
                                     C, true, M, w + L.q, as_stream(stream), {}, true),
                "ttq_qgemm_adapters launch"))
            return e;
        const int parts = ttq::qgemv_gs_slices(T, K, M);
        if (parts > 1) ci = {w + L.q, true, M, parts, T * M};
    } else if (ttq_status e = ttq_qgemm(X, xt, T, K, ldx, s, codes, scale_f16, zero_f16, M, bits, group, C, TTQ_F32, M,
                                        w + L.q, ws_qgemm(T, K, M), stream)) {
        return e;
    }
    return device_status(ttq::launch_adapters(X, xf32, T, K, ldx, adapter_table(ad), ci, M, Y, yt == TTQ_F32, ldy,
                                              (float*)(w + L.z), as_stream(stream)),
                         "ttq_qgemm_adapters launch");
}

}  // extern "C"

// ------------------------------------------- 8-bit integers, sorted tokens

namespace {

constexpr int64_t kMaxKI8 = (int64_t)1 << 17;     // 127^2 K fits in int32
constexpr int64_t kMaxLdI8 = (int64_t)1 << 22;    // 256 rows lie within one buffer descriptor
constexpr int64_t kMaxSlots = (int64_t)1 << 30;
constexpr int64_t kMaxMoeI8Slots = (int64_t)1 << 24;

ttq_status check_k_i8(const char* name, int64_t K) {
    TTQ_REQUIRE(K > 0 && K <= kMaxKI8 && K % 16 == 0, "%s must be a positive multiple of 16, at most 2^17", name);
    return TTQ_OK;
}

ttq_status check_codes(const char* name, const void* p, int64_t rows, int64_t K, int64_t ld) {
    TTQ_REQUIRE(ld >= K && ld <= kMaxDim && ld % 16 == 0,
                "%s: row stride %lld is below the row length or not a multiple of 16", name, (long long)ld);
    TTQ_REQUIRE(rows == 0 || (p != nullptr && aligned(p, 16)), "%s: null or not 16-byte aligned", name);
    return TTQ_OK;
}

ttq_status check_words(const char* name, const void* p) {
    TTQ_REQUIRE(p != nullptr && aligned(p, 4), "%s: null or misaligned", name);
    return TTQ_OK;
}

// The product's arguments (X is checked by the caller).
ttq_status check_product_i8(int64_t T, int64_t K, int64_t M, const int8_t* W, const float* w_scale, int64_t ldw,
                            const void* Y, int yt, int64_t ldy) {
    TTQ_REQUIRE(dim_ok(T) && dim_ok(M), "T or M out of range");
    if (ttq_status e = check_k_i8("K", K)) return e;
    if (ttq_status e = check_codes("W", W, T == 0 ? 0 : M, K, ldw)) return e;
    if (ttq_status e = check_output(Y, yt, T, M, ldy)) return e;
    if (T > 0 && M > 0)
        if (ttq_status e = check_words("w_scale", w_scale)) return e;
    if (ldw > kMaxLdI8) return fail(TTQ_ERR_UNSUPPORTED, "W: row stride above 2^22");
    if (!ttq::i8_product_fits(T, M, 0)) return fail(TTQ_ERR_UNSUPPORTED, "T x M is beyond one launch");
    return TTQ_OK;
}

size_t ws_qgemm_i8_codes(int64_t T, int64_t K) { return round_up((size_t)T * K); }
size_t ws_qgemm_i8_head(int64_t T, int64_t K) { return ws_qgemm_i8_codes(T, K) + round_up((size_t)T * 4); }

ttq_status check_rows_moe(const char* name, const void* p, int t, int64_t rows, int64_t K, int64_t ld) {
    TTQ_REQUIRE(dim_ok(rows), "rows out of range");
    return check_matrix(name, p, t, rows, K, ld);
}

ttq_status check_slots(int64_t T, int64_t topk) {
    TTQ_REQUIRE(dim_ok(T), "T out of range");
    TTQ_REQUIRE(topk >= 1 && topk <= ttq::kRouteMaxTopk, "topk must be in [1, %d]", ttq::kRouteMaxTopk);
    TTQ_REQUIRE(T * topk <= kMaxSlots, "T * topk above 2^30");
    return TTQ_OK;
}

ttq_status check_experts_i8(const char* name, const ttq_expert_i8& q, int64_t K) {
    TTQ_REQUIRE(q.s != nullptr && aligned(q.s, 16), "%s.s: null or not 16-byte aligned", name);
    TTQ_REQUIRE(q.s_stride == 0 || (q.s_stride >= K && q.s_stride % 4 == 0 && q.s_stride <= kMaxDim),
                "%s.s_stride: neither 0 nor a multiple of 4 of at least the row length", name);
    TTQ_REQUIRE(q.codes != nullptr && aligned(q.codes, 16), "%s.codes: null or not 16-byte aligned", name);
    TTQ_REQUIRE(q.scale != nullptr && aligned(q.scale, 4), "%s.scale: null or misaligned", name);
    return TTQ_OK;
}

ttq_status check_moe_i8_sizes(int64_t T, int64_t topk, int64_t K, int64_t I, int64_t M, int64_t E) {
    if (ttq_status e = check_slots(T, topk)) return e;
    TTQ_REQUIRE(E >= 1 && E <= ttq::kMoeMaxExperts, "E (experts) must be in [1, %d]", ttq::kMoeMaxExperts);
    TTQ_REQUIRE(dim_ok(M), "M out of range");
    if (ttq_status e = check_k_i8("K", K)) return e;
    if (ttq_status e = check_k_i8("I", I)) return e;
    if (2 * I * K >= kMaxExpertBytes || M * I >= kMaxExpertBytes)
        return fail(TTQ_ERR_UNSUPPORTED, "an expert's codes take 2 GiB or more");
    if (T * topk > kMaxMoeI8Slots || T * K >= kMaxExpertBytes)
        return fail(TTQ_ERR_UNSUPPORTED, "more than 2^24 slots, or 2 GiB of the tokens' codes: pass the tokens in chunks");
    if (!ttq::i8_product_fits(T * topk, I > M ? I : M, E))
        return fail(TTQ_ERR_UNSUPPORTED, "slots x channels is beyond one launch");
    return TTQ_OK;
}

}  // namespace

extern "C" {

ttq_status ttq_quantize_rows(const void* X, int xt, int64_t R, int64_t K, int64_t ldx, const float* s, int divide,
                             int8_t* codes, int64_t ldc, float* scale, void* stream) {
    g_last_error.clear();
    TTQ_REQUIRE(dim_ok(R), "R out of range");
    if (ttq_status e = check_k_i8("K", K)) return e;
    if (ttq_status e = check_matrix("X", X, xt, R, K, ldx)) return e;
    TTQ_REQUIRE(aligned(s, 16), "s: pointer not 16-byte aligned");
    if (ttq_status e = check_codes("codes", codes, R, K, ldc)) return e;
    if (R == 0) return TTQ_OK;
    if (ttq_status e = check_words("scale", scale)) return e;
    return device_status(ttq::launch_quantize_rows({X, xt == TTQ_F32, ldx, R, K, s, divide != 0, codes, ldc, scale},
                                                   as_stream(stream)),
                         "ttq_quantize_rows launch");
}

size_t ttq_gemm_i8_workspace_bytes(int64_t T, int64_t K, int64_t M) {
    if (!dim_ok(T) || !dim_ok(M) || K <= 0 || K > kMaxKI8 || K % 16 || !ttq::i8_product_fits(T, M, 0)) return 0;
    return round_up(ttq::i8_product_ws_bytes(T, K, M)) + kAlign;
}

ttq_status ttq_gemm_i8(const int8_t* X, const float* x_scale, int64_t T, int64_t K, int64_t ldx, const int8_t* W,
                       const float* w_scale, int64_t M, int64_t ldw, void* Y, int yt, int64_t ldy, void* ws,
                       size_t ws_bytes, void* stream) {
    g_last_error.clear();
    if (ttq_status e = check_product_i8(T, K, M, W, w_scale, ldw, Y, yt, ldy)) return e;
    if (ttq_status e = check_codes("X", X, M == 0 ? 0 : T, K, ldx)) return e;
    if (ldx > kMaxLdI8) return fail(TTQ_ERR_UNSUPPORTED, "X: row stride above 2^22");
    if (T == 0 || M == 0) return TTQ_OK;
    if (ttq_status e = check_words("x_scale", x_scale)) return e;
    if (ttq_status e = check_ws(ws, ws_bytes, ttq_gemm_i8_workspace_bytes(T, K, M))) return e;
    return device_status(ttq::launch_i8_product({X, ldx, x_scale, T, K, W, ldw, w_scale, M, Y, ldy}, yt == TTQ_F32, ws,
                                                as_stream(stream)),
                         "ttq_gemm_i8 launch");
}

size_t ttq_qgemm_i8_workspace_bytes(int64_t T, int64_t K, int64_t M) {
    const size_t n = ttq_gemm_i8_workspace_bytes(T, K, M);
    return n == 0 ? 0 : ws_qgemm_i8_head(T, K) + n;
}

ttq_status ttq_qgemm_i8(const void* X, int xt, int64_t T, int64_t K, int64_t ldx, const float* s, const int8_t* W,
                        const float* w_scale, int64_t M, int64_t ldw, void* Y, int yt, int64_t ldy, void* ws,
                        size_t ws_bytes, void* stream) {
    g_last_error.clear();
    if (ttq_status e = check_product_i8(T, K, M, W, w_scale, ldw, Y, yt, ldy)) return e;
    if (ttq_status e = check_matrix("X", X, xt, M == 0 ? 0 : T, K, ldx)) return e;
    TTQ_REQUIRE(aligned(s, 16), "s: pointer not 16-byte aligned");
    if (T == 0 || M == 0) return TTQ_OK;
    if (ttq_status e = check_ws(ws, ws_bytes, ttq_qgemm_i8_workspace_bytes(T, K, M))) return e;
    char* w = (char*)ws;
    int8_t* q = (int8_t*)w;
    float* qs = (float*)(w + ws_qgemm_i8_codes(T, K));
    hipStream_t st = as_stream(stream);
    const ttq::I8RowsArgs rows{X, xt == TTQ_F32, ldx, T, K, s, true, q, K, qs};
    const ttq::I8Product p{q, K, qs, T, K, W, ldw, w_scale, M, Y, ldy};
    if (ttq::i8_one_fits(T, K))
        return device_status(ttq::launch_i8_one(rows, p, yt == TTQ_F32, st), "ttq_qgemm_i8 launch");
    if (ttq_status e = device_status(ttq::launch_quantize_rows(rows, st), "ttq_qgemm_i8 launch")) return e;
    return device_status(ttq::launch_i8_product(p, yt == TTQ_F32, w + ws_qgemm_i8_head(T, K), st), "ttq_qgemm_i8 launch");
}

size_t ttq_moe_sort_workspace_bytes(int64_t T, int64_t topk, int64_t E) {
    if (!dim_ok(T) || topk < 1 || topk > ttq::kRouteMaxTopk || T * topk > kMaxSlots || E < 1 || E > ttq::kMoeMaxExperts)
        return 0;
    return round_up(ttq::moe_sort_ws_bytes(T * topk, E));
}

ttq_status ttq_moe_sort(const int32_t* ids, int64_t T, int64_t topk, int64_t E, int32_t* offsets, int32_t* order,
                        int32_t* pos, void* ws, size_t ws_bytes, void* stream) {
    g_last_error.clear();
    if (ttq_status e = check_slots(T, topk)) return e;
    TTQ_REQUIRE(E >= 1 && E <= ttq::kMoeMaxExperts, "E (experts) must be in [1, %d]", ttq::kMoeMaxExperts);
    if (ttq_status e = check_words("offsets", offsets)) return e;
    if (T > 0) {
        if (ttq_status e = check_words("ids", ids)) return e;
        if (ttq_status e = check_words("order", order)) return e;
        if (ttq_status e = check_words("pos", pos)) return e;
        if (ttq_status e = check_ws(ws, ws_bytes, ttq_moe_sort_workspace_bytes(T, topk, E))) return e;
    }
    return device_status(ttq::launch_moe_sort(ids, T * topk, (int)E, offsets, order, pos, (int32_t*)ws, as_stream(stream)),
                         "ttq_moe_sort launch");
}

ttq_status ttq_moe_gather(const void* X, int xt, int64_t T, int64_t K, int64_t ldx, const int32_t* pos, int64_t topk,
                          void* R, int64_t rows, int64_t ldr, void* stream) {
    g_last_error.clear();
    if (ttq_status e = check_slots(T, topk)) return e;
    TTQ_REQUIRE(K > 0 && K <= kMaxDim, "K out of range");
    if (ttq_status e = check_matrix("X", X, xt, T, K, ldx)) return e;
    if (ttq_status e = check_rows_moe("R", R, xt, T == 0 ? 0 : rows, K, ldr)) return e;
    if (T == 0 || rows == 0) return TTQ_OK;
    if (ttq_status e = check_words("pos", pos)) return e;
    return device_status(ttq::launch_moe_gather(X, (int)esize(xt), T, K, ldx, pos, (int)topk, R, rows, ldr,
                                                as_stream(stream)),
                         "ttq_moe_gather launch");
}

ttq_status ttq_moe_combine(const void* R, int rt, int64_t rows, int64_t ldr, const int32_t* pos, const float* w,
                           int64_t T, int64_t topk, int64_t M, void* Y, int yt, int64_t ldy, void* stream) {
    g_last_error.clear();
    if (ttq_status e = check_slots(T, topk)) return e;
    TTQ_REQUIRE(dim_ok(M), "M out of range");
    if (ttq_status e = check_rows_moe("R", R, rt, T == 0 || M == 0 ? 0 : rows, M, ldr)) return e;
    if (ttq_status e = check_output(Y, yt, T, M, ldy)) return e;
    if (T == 0 || M == 0) return TTQ_OK;
    if (ttq_status e = check_words("pos", pos)) return e;
    TTQ_REQUIRE(aligned(w, 4), "w: misaligned");
    return device_status(ttq::launch_moe_combine(R, rt == TTQ_F32, rows, ldr, pos, w, T, (int)topk, M, Y, yt == TTQ_F32,
                                                 ldy, as_stream(stream)),
                         "ttq_moe_combine launch");
}

ttq_status ttq_moe_combine_grad(const void* dY, int yt, int64_t T, int64_t M, int64_t lddy, const void* R, int rt,
                                int64_t rows, int64_t ldr, const int32_t* pos, const float* w, int64_t topk, void* dR,
                                int64_t lddr, float* dw, void* stream) {
    g_last_error.clear();
    if (ttq_status e = check_slots(T, topk)) return e;
    TTQ_REQUIRE(M > 0 && dim_ok(M), "M out of range");
    if (ttq_status e = check_matrix("dY", dY, yt, T, M, lddy)) return e;
    TTQ_REQUIRE(dtype_ok(rt), "R: unknown dtype %d", rt);
    TTQ_REQUIRE(dim_ok(rows), "rows out of range");
    if (T > 0 && dw != nullptr)
        if (ttq_status e = check_rows_moe("R", R, rt, rows, M, ldr)) return e;
    if (T > 0 && dR != nullptr)
        if (ttq_status e = check_rows_moe("dR", dR, rt, rows, M, lddr)) return e;
    TTQ_REQUIRE(dR == nullptr || dR != R, "dR must not be R");
    TTQ_REQUIRE(aligned(w, 4) && aligned(dw, 4), "w or dw: misaligned");
    if (T == 0 || (dR == nullptr && dw == nullptr)) return TTQ_OK;
    if (ttq_status e = check_words("pos", pos)) return e;
    return device_status(ttq::launch_moe_combine_grad(dY, yt == TTQ_F32, lddy, R, rt == TTQ_F32, rows, ldr, pos, w, T,
                                                      (int)topk, M, dR, lddr, dw, as_stream(stream)),
                         "ttq_moe_combine_grad launch");
}

size_t ttq_moe_i8_workspace_bytes(int64_t T, int64_t topk, int64_t K, int64_t I, int64_t M, int64_t E) {
    if (check_moe_i8_sizes(T, topk, K, I, M, E)) return 0;
    return ttq::moe_i8_ws_bytes(T, topk, K, I, M, E) + kAlign;
}

ttq_status ttq_moe_i8(const ttq_moe_i8_args* a, void* ws, size_t ws_bytes, void* stream) {
    g_last_error.clear();
    TTQ_REQUIRE(a != nullptr, "args: null pointer");
    if (ttq_status e = check_moe_i8_sizes(a->T, a->topk, a->K, a->I, a->M, a->E)) return e;
    TTQ_REQUIRE(a->act == TTQ_ACT_SILU || a->act == TTQ_ACT_GELU_TANH, "act: unknown value %d", a->act);
    if (ttq_status e = check_matrix("X", a->X, a->xt, a->T, a->K, a->ldx)) return e;
    if (ttq_status e = check_output(a->Y, a->yt, a->T, a->M, a->ldy)) return e;
    if (a->T == 0 || a->M == 0) return TTQ_OK;
    TTQ_REQUIRE(a->ids != nullptr && aligned(a->ids, 4) && a->w != nullptr && aligned(a->w, 4),
                "ids or w: null or misaligned");
    if (ttq_status e = check_experts_i8("gate_up", a->gate_up, a->K)) return e;
    if (ttq_status e = check_experts_i8("down", a->down, a->I)) return e;
    if (ttq_status e = check_ws(ws, ws_bytes, ttq::moe_i8_ws_bytes(a->T, a->topk, a->K, a->I, a->M, a->E))) return e;
    return device_status(ttq::launch_moe_i8(a, (char*)ws, as_stream(stream)), "ttq_moe_i8 launch");
}

}  // extern "C"
