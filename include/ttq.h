/*
 * libttq — activation-aware test-time quantization (TTQ) of one linear layer,
 * per prompt, on AMD MI355X (gfx950).
 *
 * Source of the method: the nubint.ai review page "TTQ: Activation-Aware
 * Test-Time Quantization to Accelerate LLM Inference On The Fly", section
 * "proposed method" (bullets b1..b7).  "[TTQ §method b3]" below means its
 * third bullet.
 *
 * Conventions shared by every call
 * --------------------------------
 *  - Shapes: T tokens, K input channels, M output channels.
 *    X is [T][K] row-major with row stride ldx (elements),
 *    W is [M][K] row-major with row stride ldw (the Linear weight layout),
 *    Y is [T][M] row-major with row stride ldy.
 *  - Every pointer is DEVICE memory, allocated and owned by the caller; the
 *    library allocates nothing and never synchronises.  Every call only
 *    enqueues kernels on `stream` (a hipStream_t; NULL = the null stream)
 *    and returns; results are ready when the stream reaches that point.
 *    Global state: the calling thread's last error text, and a per-device
 *    memo of kernel residency queried from the runtime once (a property of
 *    the code object: it never changes a result).  Calls are safe from any
 *    thread and on any stream.
 *  - Packed codes: for each output row, the K codes form a little-endian bit
 *    stream (code j occupies stream bits [bits*j, bits*j + bits), least
 *    significant bit first; stream bit i is bit i%32 of int32 word i/32).
 *    codes is dense: [M][K*bits/32] int32.
 *  - Per-group step and zero point: fp16 bit patterns, dense [M][K/group];
 *    the group of channel j is j / group (consecutive input channels of one
 *    output row).  The zero point is an integer stored as fp16.
 *  - Argument checks run on the host before any HIP call.  A failed check
 *    returns TTQ_ERR_INVALID (or TTQ_ERR_UNSUPPORTED for well-formed but
 *    unimplemented options) and launches nothing.  A failed launch returns
 *    TTQ_ERR_DEVICE.  Faults during execution surface at the caller's next
 *    synchronisation.  After a non-OK status the outputs are undefined.
 *    ttq_last_error() describes the last non-OK status of the calling thread.
 *  - Alignment: X, W and codes base pointers 16-byte aligned and the X/W row
 *    strides a multiple of 16 bytes; Y aligned to its element size, any row
 *    stride >= M; s 16-byte aligned; ssq 8-byte aligned; workspace 256-byte
 *    aligned.
 *  - Limits: K a positive multiple of 32 (of 8 for ttq_stats), at most 2^18;
 *    T, M and row strides at most 2^30; bits in
 *    {2,3,4,5}; group in {16,32,64,128} dividing K; 0 <= rank <= 64
 *    (ttq_lowrank_factors: rank <= l <= 32).
 *    T == 0 or M == 0 is a valid empty call (nothing is launched, except
 *    that ttq_stats with accumulate == 0 still zeroes ssq).
 *  - Inputs are expected to be finite.  The quantizer gives a NaN weight
 *    code 0 and leaves it out of its group's range; other non-finite inputs
 *    give unspecified (but memory-safe) outputs.
 */
#ifndef TTQ_H
#define TTQ_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    TTQ_OK = 0,
    TTQ_ERR_INVALID = 1,      /* malformed arguments: nothing launched      */
    TTQ_ERR_UNSUPPORTED = 2,  /* well-formed but not implemented            */
    TTQ_ERR_DEVICE = 3        /* the HIP runtime refused a launch           */
} ttq_status;

typedef enum {
    TTQ_F32 = 0,              /* IEEE binary32                              */
    TTQ_BF16 = 1              /* bfloat16 (upper half of a binary32)        */
} ttq_dtype;

/*
 * ttq_stats — per-channel sum of squares of the prompt's activations.
 * [TTQ §method b2, b3]: the diagonal of the input covariance, estimated
 * online from the prompt itself.
 *   ssq[j] (+)= sum_{t<T} X[t][j]^2, accumulated in fp64.
 *   X: [T][K] fp32 or bf16 (xt), stride ldx >= K.   ssq: [K] fp64, output.
 *   accumulate != 0 adds to the existing ssq (chunked prefill), else
 *   overwrites it.  ws, ws_bytes: unused (the reduction runs in one
 *   kernel without partial sums in memory); any value, NULL included.
 *   All sums are reduced in a fixed order, so results are bitwise
 *   reproducible run to run.  K must be a multiple of 8.
 */
ttq_status ttq_stats(const void* X, int xt, int64_t T, int64_t K, int64_t ldx,
                     double* ssq, int accumulate, void* ws, size_t ws_bytes,
                     void* stream);

/*
 * ttq_stats_p — per-channel sum of |x|^p, for a moment order p fixed in
 * advance.  [TTQ §method b4]: alpha, lambda and p are fixed, not searched;
 * p = 2 is the diagonal covariance of ttq_stats, p = 1 the mean absolute
 * activation of the original AWQ statistic.
 *   msum[j] (+)= sum_{t<T} |X[t][j]|^p in fp64: exact squares for p = 2,
 *   exact |x| for p = 1, fp64 pow(|x|, p) otherwise (0 for x = 0).
 *   p finite and > 0 (else TTQ_ERR_INVALID).  Everything else (X, msum,
 *   accumulate, ws, ordering and reproducibility) is as for ttq_stats, which
 *   is this call with p = 2.  Feed msum to ttq_awq_scales with the same p.
 */
ttq_status ttq_stats_p(const void* X, int xt, int64_t T, int64_t K, int64_t ldx,
                       float p, double* msum, int accumulate, void* ws,
                       size_t ws_bytes, void* stream);

/*
 * ttq_awq_scales — shrunk AWQ per-channel scales.
 * [TTQ §method b2-b4]: c = ssq / n_tokens; lambda = lambda_rel * mean(c)
 * (shrinkage C + lambda I); s[j] = (c[j] + lambda)^(alpha / p), evaluated in
 * fp64 and rounded once to fp32; s[j] = 1 where c[j] + lambda == 0.
 * alpha, lambda_rel, p are fixed in advance (no search).
 *   ssq: [K] fp64 input, the sums of |x|^p from ttq_stats_p with the same p
 *   (sums of squares for p = 2).  s: [K] fp32 output.  n_tokens > 0.
 *   alpha and lambda_rel finite and >= 0; p finite and > 0.
 */
ttq_status ttq_awq_scales(const double* ssq, int64_t n_tokens, int64_t K,
                          float alpha, float lambda_rel, float p, float* s,
                          void* stream);

/*
 * ttq_quantize_groups — group-wise RTN of the scaled (residual) weight.
 * [TTQ §method b1] group-wise RTN; [TTQ §method b2] the weight is scaled by
 * s per input channel; [TTQ §method b5] with low-rank factors the residual
 * W - B A is quantized.
 *   v[o][j] = fp32( (W[o][j] - sum_{k<rank} B[o][k] A[k][j]) * s[j] ), the
 *     residual accumulated in fp64 in rank order; without factors this is
 *     the correctly rounded fp32 product W*s.
 *   Per group: mn = min(0, min v), mx = max(0, max v);
 *     step = fp16 rounded up of fp32(mx - mn) / (2^bits - 1) (1 if zero);
 *     zero = clamp(rne(-mn / step), 0, 2^bits - 1);
 *     code = clamp(rne(v / step) + zero, 0, 2^bits - 1).
 *   W: [M][K] fp32/bf16 (wt), stride ldw.  s: [K] fp32, or NULL for s = 1.
 *   B: [M][rank] fp32 dense, A: [rank][K] fp32 dense; both NULL iff rank 0.
 *   Outputs: codes [M][K*bits/32], scale_f16 and zero_f16 [M][K/group].
 *   Codes whose v/step lies within ~1e-5 of a step of a rounding boundary
 *   may differ from an exact-division evaluation (v * (1/step) is used).
 */
ttq_status ttq_quantize_groups(const void* W, int wt, int64_t M, int64_t K, int64_t ldw,
                               const float* s, int bits, int group,
                               const float* B, const float* A, int rank,
                               int32_t* codes, uint16_t* scale_f16, uint16_t* zero_f16,
                               void* stream);

/*
 * ttq_qgemm — the quantized projection Y = W_hat (X / s).
 * [TTQ §method b7] quantized projection kernel; [TTQ §method b1] QDQ:
 * W_hat[o][j] = (code - zero) * step; [TTQ §method b2] inputs divided by s.
 *   Y[t][o] = sum_j W_hat[o][j] * X[t][j] / s[j].
 *   For T >= 5 the dequantized weight (code - zero) * step / s[j] is
 *   rounded once to bf16 and multiplied with X on the matrix cores with fp32
 *   accumulation (bf16 X is used as is; fp32 X is split into two bf16 halves
 *   and the weight too, three products, for near-fp32 accuracy).
 *   X: [T][K] (xt), s: [K], codes/scale/zero as produced by
 *   ttq_quantize_groups for (M, K, bits, group).  Y: [T][M] fp32 or bf16
 *   (yt), overwritten.  Y must not overlap any input.
 *   Execution paths: for T <= 4 with K a multiple of 128 (decode steps) the
 *   vector ALUs compute step * (sum code * x/s - zero * sum x/s) per group
 *   in fp32, with no bf16 rounding; for bf16 X with 5 <= T <= 16, 4-bit
 *   codes, groups of 32, 64 or 128 and K a multiple of 128 the matrix cores
 *   compute the same per-group sums with x * (1/s) rounded once to bf16
 *   (formed in LDS by the same launch, with its 32-channel sums) and each
 *   code taken exactly as the bf16 number 128 + code (K split over
 *   workgroups of 64 rows: fp32 partials in ws, added in slice order by a
 *   second kernel); otherwise, for 5 <= T <= 128 with K a multiple
 *   of 128 (at most 16384) the codes stream straight into registers and are
 *   expanded there to the bf16 weights above; for bf16 X with T >= 192 and
 *   K a multiple of 64 the weight is dequantized once into ws (M*K bf16) and
 *   multiplied by a matrix-core GEMM; otherwise codes are dequantized tile
 *   by tile inside the GEMM kernel.  The last three see bitwise the same
 *   bf16 weights.
 *   For bf16 X with 12 <= T <= 16 (where the sums path does not apply) the
 *   expansion runs split over K (each workgroup: 64 rows, one K slice; fp32
 *   partials in ws, added in slice order by a second kernel).  The T >= 192
 *   GEMM also runs as two K slices when its 128 x 256 output tiles number
 *   fewer than 192 and K >= 8192 (a multiple of 128): fp32 partial products
 *   in ws, then Y = P0 + P1.
 *   ws: at least ttq_workspace_bytes(T, K, M, bits, group, 0) bytes (for
 *   5 <= T <= 16 and K a multiple of 128: the larger of S*T*M*4 for the
 *   S K slices of the sums path (whole 512-channel sets, at most 8 a slice,
 *   S*ceil(M/64) about 256; none when S = 1) and, when T >= 12, the split
 *   partials S'*T*M*4 for S' <= K/128 slices; M*K*2 when T >= 192, plus 2*T*M'*4 with M' = M
 *   rounded up to 4 when the GEMM runs as two K slices; each part rounded up
 *   to 256; none otherwise); only read and written by the kernels this call
 *   enqueues.
 */
ttq_status ttq_qgemm(const void* X, int xt, int64_t T, int64_t K, int64_t ldx,
                     const float* s, const int32_t* codes, const uint16_t* scale_f16,
                     const uint16_t* zero_f16, int64_t M, int bits, int group,
                     void* Y, int yt, int64_t ldy, void* ws, size_t ws_bytes,
                     void* stream);

/*
 * ttq_qgemm_batched — one decode step of P prompts in one launch.
 * [TTQ §method b7] the quantized projection, for several prompts at once:
 * every prompt has its own quantized state (its own s, codes, steps and
 * zeros: TTQ quantizes per prompt), so this is P independent projections
 * sharing one launch.  Prompt p uses
 *   X + p*x_stride ([T][K], stride ldx, elements of xt), s + p*s_stride,
 *   codes + p*codes_stride (int32 words), scale_f16/zero_f16 + p*sz_stride,
 *   Y + p*y_stride ([T][M], stride ldy, elements of yt),
 * and gets exactly what ttq_qgemm gives for it alone (the same kernel, bit
 * for bit).  1 <= T <= 4, K a multiple of 128, 1 <= P <= 65535; strides
 * >= 0, keeping every prompt's X, s and codes 16-byte aligned; prompts'
 * X and Y regions must not overlap.  No workspace.
 */
ttq_status ttq_qgemm_batched(const void* X, int xt, int64_t P, int64_t T, int64_t K, int64_t ldx,
                             int64_t x_stride, const float* s, int64_t s_stride,
                             const int32_t* codes, int64_t codes_stride,
                             const uint16_t* scale_f16, const uint16_t* zero_f16, int64_t sz_stride,
                             int64_t M, int bits, int group, void* Y, int yt, int64_t ldy,
                             int64_t y_stride, void* stream);

/*
 * ttq_lowrank_add — Y += B (A X), the dynamic low-rank term.
 * [TTQ §method b5]: W = W_q + B A, so the layer adds B (A X) to the
 * quantized projection.  Computed in fp32: Z[t][k] = sum_j A[k][j] X[t][j],
 * then Y[t][o] += sum_k B[o][k] Z[t][k].
 *   X: [T][K] (xt), A: [rank][K] fp32, B: [M][rank] fp32, Y: [T][M] (yt),
 *   updated in place.  ws: at least ttq_workspace_bytes(T, K, M, 2, 32, rank).
 */
ttq_status ttq_lowrank_add(const void* X, int xt, int64_t T, int64_t K, int64_t ldx,
                           const float* A, const float* B, int64_t M, int rank,
                           void* Y, int yt, int64_t ldy, void* ws, size_t ws_bytes,
                           void* stream);

/*
 * ttq_lowrank_factors — the dynamic low-rank factors of one prompt.
 * [TTQ §method b5]: W = W_q + B A with factors formed per prompt.  The top
 * `rank` factors of W diag(s) (s from this prompt's ttq_awq_scales) are
 * estimated by randomized subspace iteration (Halko, Martinsson and Tropp,
 * "Finding structure with randomness", 2011): with A_s = W diag(s),
 *   Q = orth(A_s omega^T);  q times: Q = orth(A_s orth(A_s^T Q));
 *   Q^T A_s = U~ S V^T;  B = Q U~_r S_r,  A = V_r^T diag(1/s),
 * so that B A approximates W and B (A X) acts on the raw input; feed them
 * to ttq_quantize_groups / ttq_linear with the same s.  orth() is a
 * Cholesky QR with an fp64 Gram matrix; the inner orth of each power
 * iteration is omitted (orth(A_s orth(A_s^T Q)) = orth(A_s A_s^T Q) exactly,
 * the inner orth being a right product with an upper triangular matrix of
 * positive diagonal); the passes over W run on the matrix cores with fp32
 * accuracy; the small eigenproblem is a fp64 Jacobi iteration.
 *   W: [M][K] bf16 (wt; fp32 W returns TTQ_ERR_UNSUPPORTED), stride ldw,
 *   K a multiple of 32.  s: [K] fp32.  omega: [l][K] fp32, the caller's
 *   Gaussian test vectors (one per row), 1 <= rank <= l <= 32, l <= M, K.
 *   q: power iterations, 0..64.  Outputs B: [M][rank] fp32, A: [rank][K]
 *   fp32, dense.  Singular vectors are determined up to sign (and within
 *   repeated singular values); B A is the unique part.  A zero weight gives
 *   zero factors.  ws: ttq_lowrank_factors_workspace_bytes(M, K, l) bytes,
 *   256-byte aligned (it holds a bf16 transpose of W); results are bitwise
 *   reproducible run to run.
 */
ttq_status ttq_lowrank_factors(const void* W, int wt, int64_t M, int64_t K, int64_t ldw,
                               const float* s, const float* omega, int l, int q, int rank,
                               float* B, float* A, void* ws, size_t ws_bytes, void* stream);

/* Workspace bytes for ttq_lowrank_factors (0 for sizes it does not accept). */
size_t ttq_lowrank_factors_workspace_bytes(int64_t M, int64_t K, int l);

/*
 * Workspace size (bytes) sufficient for every call above and for ttq_linear
 * with these sizes (including the intermediate ssq, s, codes, steps and
 * zeros that ttq_linear keeps there when the caller does not supply them).
 * Returns 0 for arguments that no call accepts.
 */
size_t ttq_workspace_bytes(int64_t T, int64_t K, int64_t M, int bits, int group, int rank);

/*
 * ttq_linear — the whole per-prompt path of one linear layer.
 * [TTQ §method b1-b5, b7]: statistics of this prompt's X (sums of |x|^p,
 * ttq_stats_p) -> shrunk AWQ scales with the same p -> group RTN of
 * (W - B A) diag(s) -> quantized projection, plus B (A X) when rank > 0.
 * Equivalent to the five calls above in order.
 * The optional outputs (ssq, s, codes, scale_f16, zero_f16) receive the
 * prompt's quantization state so that later decode steps can call ttq_qgemm
 * on it; when NULL they live in the workspace.
 * Execution: statistics (the reduction also forms lambda), then one
 * quantizer pass that evaluates s for its channels (same arithmetic as
 * ttq_awq_scales), writes codes, steps and zeros, and for bf16 X with
 * T >= 192 and K a multiple of 64 also the dequantized weight into ws, which
 * the matrix-core GEMM then multiplies (otherwise the fused kernel of
 * ttq_qgemm runs); then the low-rank term.
 * stage_events: NULL, or TTQ_LINEAR_STAGE_EVENTS hipEvent_t handles created
 * by the caller: a (start, stop) pair for each of the statistics, the
 * quantizer, the projection and the low-rank term, in that order.  The
 * stage's first kernel stamps `start` when it starts and its last kernel
 * stamps `stop` when it ends (kernel timestamps: nothing extra is enqueued);
 * a stage that launches nothing (the low-rank term when rank == 0) records
 * both on `stream` as markers.  For per-stage timing; never blocks.
 */
#define TTQ_LINEAR_STAGE_EVENTS 8
typedef struct ttq_linear_args {
    const void* X;  int xt;  int64_t T;  int64_t K;  int64_t ldx;
    const void* W;  int wt;  int64_t M;  int64_t ldw;
    float alpha;  float lambda_rel;  float p;
    int bits;  int group;
    const float* B;  const float* A;  int rank;
    void* Y;  int yt;  int64_t ldy;
    double* ssq;  float* s;  int32_t* codes;  uint16_t* scale_f16;  uint16_t* zero_f16;
    void* const* stage_events;
} ttq_linear_args;

ttq_status ttq_linear(const ttq_linear_args* args, void* ws, size_t ws_bytes, void* stream);

/*
 * ttq_linear_shared — several layers that read the same X (q, k and v; gate
 * and up), with one statistics pass for all of them.
 * [TTQ §method b3]: the statistics are those of the layer input X, so
 * projections of the same input share them (and hence lambda and s).
 *   layers[0..n-1], 1 <= n <= 64: ttq_linear arguments that agree in X, xt,
 *   T, K, ldx, alpha, lambda_rel and p; M, W, bits, group, the low-rank
 *   factors, Y and the state outputs are per layer.  The statistics are
 *   reduced once (into layers[0].ssq if given; every other ssq must be
 *   NULL), then each layer runs the quantizer and projection of ttq_linear
 *   in order, with results bitwise equal to separate ttq_linear calls.
 *   stage_events must be NULL.  ws: ttq_linear_shared_workspace_bytes(
 *   layers, n) bytes (the statistics plus the largest layer's state and
 *   scratch; layers run one after another on the stream and reuse it).
 */
ttq_status ttq_linear_shared(const ttq_linear_args* layers, int n, void* ws, size_t ws_bytes,
                             void* stream);

/* Workspace bytes for ttq_linear_shared (0 when some layer's sizes are not accepted). */
size_t ttq_linear_shared_workspace_bytes(const ttq_linear_args* layers, int n);

/*
 * ttq_linear_noalloc — ttq_linear without a workspace argument, for callers
 * that cannot allocate device memory: code under HIP graph capture, tight
 * serving loops, harnesses that forbid hipMalloc.  The library allocates
 * nothing here either: the workspace is a device array inside the library,
 * TTQ_NOALLOC_SCRATCH_BYTES (64 MiB) on each GPU it runs on, held until the
 * process ends.  Arguments, results and the other checks are those of
 * ttq_linear; a layer whose ttq_workspace_bytes(T, K, M, bits, group, rank)
 * exceeds TTQ_NOALLOC_SCRATCH_BYTES returns TTQ_ERR_INVALID (give the state
 * outputs ssq, s, codes, scale_f16, zero_f16 to keep them out of the array).
 * Every call on a GPU shares that GPU's array: calls that overlap on one GPU
 * (on different streams, or from threads without ordering) race and give
 * undefined results.  The array's address is resolved on the first call on
 * each device (TTQ_ERR_DEVICE if that fails).
 */
#define TTQ_NOALLOC_SCRATCH_BYTES ((size_t)64 << 20)
ttq_status ttq_linear_noalloc(const ttq_linear_args* args, void* stream);

/*
 * Projections whose weights each token chooses.  [TTQ §method b7] the
 * quantized projection kernel, where the tokens of one launch do not share
 * their weights: the experts of a mixture-of-experts layer, and low-rank
 * adapters (the B A of [TTQ §method b5]) of many requests beside one shared
 * projection.
 */

typedef enum {
    TTQ_SCORE_SOFTMAX = 0,    /* exp(l) / sum of exp(l) over all experts    */
    TTQ_SCORE_SIGMOID = 1     /* 1 / (1 + exp(-l))                          */
} ttq_score;

typedef enum {
    TTQ_ACT_SILU = 0,         /* x / (1 + exp(-x))                          */
    TTQ_ACT_GELU_TANH = 1     /* x (1 + tanh(sqrt(2/pi)(x + 0.044715 x^3))) / 2 */
} ttq_act;

/*
 * ttq_moe_route — the top-k experts of each token and their weights.
 *   logits: [T][E] fp32 or bf16 (lt), row stride ldl >= E.  ids, w: [T][topk]
 *   dense.  ids[t][j] is the expert of the j-th largest logit of token t,
 *   equal logits in the order of their index; w[t][j] is its score (in fp32:
 *   softmax over all E logits, or sigmoid), divided by the sum of the topk
 *   scores if renormalize != 0.  Renormalized sigmoid scores keep their ratios
 *   below fp32's range; if the row's largest logit is below -745 they are 0.
 *   A logit that is -inf or NaN is never chosen and has score 0: where fewer
 *   than topk others are left, the remaining slots get id -1 and weight 0
 *   (all of them for a row without any).  +inf
 *   logits share the softmax equally.
 *   1 <= E <= 1024, 1 <= topk <= min(E, 32).  logits, ids and w aligned to
 *   their element size.  T == 0 is an empty call.  No workspace.
 */
ttq_status ttq_moe_route(const void* logits, int lt, int64_t T, int64_t E, int64_t ldl, int topk,
                         int score, int renormalize, int32_t* ids, float* w, void* stream);

/* Quantized state of E weights of equal shape: codes [E][rows][K*bits/32],
 * scale_f16 and zero_f16 [E][rows][K/group], dense, each expert's part as
 * ttq_quantize_groups writes it (experts that share s can be quantized in
 * one call with E*rows rows); expert e is scaled by s + e * s_stride
 * (s_stride 0: one s for all; else a multiple of 4, at least K). */
typedef struct ttq_expert_state {
    const float* s;  int64_t s_stride;
    const int32_t* codes;  const uint16_t* scale_f16;  const uint16_t* zero_f16;
} ttq_expert_state;

/*
 * ttq_moe — a gated mixture-of-experts layer on quantized experts, for few
 * tokens (decode steps; longer prompts in chunks of at most 1024 tokens).
 *   Y[t] = sum_j w[t][j] D_e (h / s_down),  h = act(g) * u,
 *   [g; u] = G_e (X[t] / s_in),  e = ids[t][j],
 *   G_e [2 I][K] and D_e [M][I] the dequantized gate_up and down weights of
 *   expert e (gate rows first), s_in and s_down their scales.
 *   X: [T][K] (xt), stride ldx.  ids, w: [T][topk] dense, e.g. from
 *   ttq_moe_route; a slot whose id is not in [0, E) adds nothing (its weight
 *   is not read), a token without any gets zeros, an expert named twice by a
 *   token counts twice.  Y: [T][M] (yt), overwritten.
 *   All sums are kept in fp32; Y is rounded once.  x / s and h enter the
 *   products with 16 bits for bf16 X and 24 for fp32 X (one or two tokens on
 *   4-bit codes in groups of 32 or more: to 2^-19 or 2^-23 of the largest of
 *   their 32 channels), codes, steps and zeros exactly.  A token's results
 *   depend on the other tokens of the call only through that choice (one or
 *   two tokens, or more) and the order of the fp32 sums.  They are
 *   reproducible run to run; an infinite or NaN x / s or h makes its token's
 *   outputs NaN and no other's.
 *   K and I multiples of 32 and of group, at most 2^18; E <= 1024;
 *   1 <= topk <= 32; T > 1024, or an expert's gate_up or down codes of 2 GiB
 *   or more, return TTQ_ERR_UNSUPPORTED.  T == 0 or M == 0 is an empty call.
 *   ws: ttq_moe_workspace_bytes(T, topk, K, I, M, E, bits, group) bytes,
 *   256-byte aligned; calls that may run at the same time need workspaces of
 *   their own.
 */
typedef struct ttq_moe_args {
    const void* X;  int xt;  int64_t T;  int64_t K;  int64_t ldx;
    const int32_t* ids;  const float* w;  int64_t topk;
    int64_t E;  int64_t I;  int64_t M;
    ttq_expert_state gate_up;  ttq_expert_state down;
    int bits;  int group;  int act;
    void* Y;  int yt;  int64_t ldy;
} ttq_moe_args;

ttq_status ttq_moe(const ttq_moe_args* args, void* ws, size_t ws_bytes, void* stream);

/* Workspace bytes for ttq_moe (0 for sizes it does not accept). */
size_t ttq_moe_workspace_bytes(int64_t T, int64_t topk, int64_t K, int64_t I, int64_t M, int64_t E,
                               int bits, int group);

/* Low-rank adapters: A [n][rank][K] and B [n][M][rank], dense, both fp32 or
 * bf16 (dt).  Adapter a uses its first r_a = clamp(ranks[a], 0, rank) rows of
 * A and columns of B (ranks NULL: all; the rest is not used) and is
 * multiplied by scale[a] (scale NULL: 1).  ids[t]: token t's adapter; an id
 * outside [0, n) means none.  1 <= rank <= 64, 0 <= n <= 65536; A and B
 * 16-byte aligned. */
typedef struct ttq_adapters {
    const void* A;  const void* B;  int dt;
    int64_t n;  int rank;
    const int32_t* ranks;  const float* scale;
    const int32_t* ids;
} ttq_adapters;

/*
 * ttq_adapters_add — each token's own low-rank adapter, added to a projection.
 * [TTQ §method b5] the term B (A X) of ttq_lowrank_add, with a (B, A) per
 * request.
 *   Y[t] = C[t] + scale_a B_a (A_a X[t]),  a = ids[t]; without an adapter
 *   Y[t] = C[t].  In fp32, rounded once to Y.
 *   X: [T][K] (xt).  C: [T][M] of Y's dtype, stride ldc, or NULL for zeros;
 *   it may be Y itself (ldc == ldy), else it must not overlap Y; Y may lie on
 *   X.  Any order of ids is accepted; runs of tokens of one adapter (prompts)
 *   cost least.
 *   K a multiple of 8, at most 2^18; ldx above 2^24 returns
 *   TTQ_ERR_UNSUPPORTED.  T == 0 or M == 0 is an empty call.
 *   ws: ttq_adapters_workspace_bytes(T, K, M, rank) bytes, 256-byte aligned.
 */
ttq_status ttq_adapters_add(const void* X, int xt, int64_t T, int64_t K, int64_t ldx,
                            const ttq_adapters* adapters, int64_t M, const void* C, int64_t ldc,
                            void* Y, int yt, int64_t ldy, void* ws, size_t ws_bytes, void* stream);

/* Workspace bytes for ttq_adapters_add (0 for sizes it does not accept). */
size_t ttq_adapters_workspace_bytes(int64_t T, int64_t K, int64_t M, int rank);

/*
 * ttq_qgemm_adapters — a quantized projection shared by the tokens' requests,
 * plus their adapters.  [TTQ §method b5, b7].
 *   Y[t] = W_hat (X[t] / s) + scale_a B_a (A_a X[t]),  a = ids[t]:
 *   ttq_qgemm followed by ttq_adapters_add, with Y rounded once, and for fp32 X
 *   with 24 bits of x / s and fp32 sums (ttq_qgemm on more than four tokens: 16
 *   bits of x and of the weight).  The arguments are those of the two calls,
 *   and K is a multiple of 32.
 *   ws: ttq_qgemm_adapters_workspace_bytes(...) bytes, 256-byte aligned.
 */
ttq_status ttq_qgemm_adapters(const void* X, int xt, int64_t T, int64_t K, int64_t ldx, const float* s,
                              const int32_t* codes, const uint16_t* scale_f16, const uint16_t* zero_f16,
                              int64_t M, int bits, int group, const ttq_adapters* adapters,
                              void* Y, int yt, int64_t ldy, void* ws, size_t ws_bytes, void* stream);

/* Workspace bytes for ttq_qgemm_adapters (0 for sizes it does not accept). */
size_t ttq_qgemm_adapters_workspace_bytes(int64_t T, int64_t K, int64_t M, int bits, int group, int rank);

/*
 * Linear layers in 8-bit integers.  [TTQ §method b1, b2, b7] the quantized
 * projection with the scaled weight W diag(s) and the input X / s both in 8
 * bits, one scale per output channel and one per token: twice the rate of the
 * bf16 matrix cores, and rows of activations that several layers share.
 *
 * 8-bit rows: codes [R][K] int8, row stride a multiple of 16 bytes, codes
 * 16-byte aligned; scale [R] fp32; row r stands for codes * scale[r].  K a
 * positive multiple of 16, at most 2^17, so that a sum of K products of codes
 * of -127..127 is exact in int32.
 * Outputs and workspaces of the calls below overlap neither each other nor an
 * input.
 */

/*
 * ttq_quantize_rows — rows of X in 8 bits.
 *   v[r][j] = X[r][j] (s NULL), fp32(X[r][j] / s[j]) (divide != 0: the input of
 *   a projection) or fp32(X[r][j] * s[j]) (divide == 0: a weight [M][K]).
 *   a = max_j |v[r][j]|;  scale[r] = fp32(a / 127), 1 where that is 0;
 *   codes[r][j] = clamp(rne(v[r][j] / scale[r]), -127, 127), the rounding of the
 *   exact quotient.
 *   A row with an infinite or NaN v gets scale NaN and codes 0, so that its
 *   products are NaN and no other row's.
 *   X: [R][K] (xt), stride ldx.  s: [K] or NULL.  codes: stride ldc >= K.
 *   R == 0 is an empty call.  No workspace.
 */
ttq_status ttq_quantize_rows(const void* X, int xt, int64_t R, int64_t K, int64_t ldx, const float* s,
                             int divide, int8_t* codes, int64_t ldc, float* scale, void* stream);

/*
 * ttq_gemm_i8 — product of 8-bit rows.
 *   Y[t][o] = x_scale[t] * w_scale[o] * sum_j X[t][j] W[o][j]: the sum exact in
 *   int32, converted to fp32 and multiplied by x_scale[t], then by w_scale[o],
 *   rounded once more to a bf16 Y.
 *   X: [T][K] int8, stride ldx;  W: [M][K] int8, stride ldw, e.g. both from
 *   ttq_quantize_rows.  Y: [T][M] (yt), stride ldy, overwritten; no overlap.
 *   ldx and ldw above 2^22, or 2^23 blocks of 256 x 256 of Y and more, return
 *   TTQ_ERR_UNSUPPORTED.  T == 0 or M == 0 is an empty call.
 *   ws: ttq_gemm_i8_workspace_bytes(T, K, M) bytes, 256-byte aligned; calls that
 *   may run at the same time need workspaces of their own.
 */
ttq_status ttq_gemm_i8(const int8_t* X, const float* x_scale, int64_t T, int64_t K, int64_t ldx, const int8_t* W,
                       const float* w_scale, int64_t M, int64_t ldw, void* Y, int yt, int64_t ldy, void* ws,
                       size_t ws_bytes, void* stream);

/* Workspace bytes for ttq_gemm_i8 (0 for sizes it does not accept). */
size_t ttq_gemm_i8_workspace_bytes(int64_t T, int64_t K, int64_t M);

/*
 * ttq_qgemm_i8 — ttq_qgemm on an 8-bit state: Y = W_hat (X / s).
 *   ttq_quantize_rows of X / s (s NULL: of X) followed by ttq_gemm_i8, with the
 *   same results.  W and w_scale: ttq_quantize_rows of the weight times s.
 *   X: [T][K] (xt), stride ldx.  The other arguments are those of ttq_gemm_i8.
 *   ws: ttq_qgemm_i8_workspace_bytes(T, K, M) bytes, 256-byte aligned.
 */
ttq_status ttq_qgemm_i8(const void* X, int xt, int64_t T, int64_t K, int64_t ldx, const float* s, const int8_t* W,
                        const float* w_scale, int64_t M, int64_t ldw, void* Y, int yt, int64_t ldy, void* ws,
                        size_t ws_bytes, void* stream);

/* Workspace bytes for ttq_qgemm_i8 (0 for sizes it does not accept). */
size_t ttq_qgemm_i8_workspace_bytes(int64_t T, int64_t K, int64_t M);

/*
 * Tokens sorted by the experts they chose, and back, for experts that multiply
 * many rows each (long prompts) and for training with them.
 */

/*
 * ttq_moe_sort — the slots (t, j) of ids [T][topk] in the order of their
 * experts, slots of one expert in the order of their index t * topk + j.
 *   offsets: [E + 1], expert e has the rows offsets[e] .. offsets[e + 1] - 1.
 *   order: [T * topk], the slot of each row, -1 behind the last row.
 *   pos: [T][topk], the row of each slot, -1 for an id outside [0, E).
 *   1 <= E <= 1024, 1 <= topk <= 32, T * topk <= 2^30; all dense int32.  T == 0
 *   writes offsets only.  ws: ttq_moe_sort_workspace_bytes(T, topk, E) bytes,
 *   256-byte aligned (0 and NULL for few slots).
 */
ttq_status ttq_moe_sort(const int32_t* ids, int64_t T, int64_t topk, int64_t E, int32_t* offsets, int32_t* order,
                        int32_t* pos, void* ws, size_t ws_bytes, void* stream);

/* Workspace bytes for ttq_moe_sort (0 also for sizes it does not accept). */
size_t ttq_moe_sort_workspace_bytes(int64_t T, int64_t topk, int64_t E);

/*
 * ttq_moe_gather — R[pos[t][j]] = X[t], the tokens' rows in their experts' order.
 *   X: [T][K] (xt), stride ldx; R: [rows][K] of the same dtype, stride ldr.  A
 *   slot whose pos is outside [0, rows) has no row; rows that no slot names are
 *   left as they were; no two slots may name one row.  K positive, any.  R
 *   16-byte aligned, its row stride a multiple of 16 bytes, no overlap with X.
 *   The gradient of X is ttq_moe_combine of R's gradient with w NULL.
 *   T == 0 or rows == 0 is an empty call.  No workspace.
 */
ttq_status ttq_moe_gather(const void* X, int xt, int64_t T, int64_t K, int64_t ldx, const int32_t* pos, int64_t topk,
                          void* R, int64_t rows, int64_t ldr, void* stream);

/*
 * ttq_moe_combine — Y[t] = sum_j w[t][j] R[pos[t][j]], the experts' rows back in
 * the tokens' order.
 *   R: [rows][M] (rt), stride ldr.  w: [T][topk] fp32, or NULL for ones.  A slot
 *   whose pos is outside [0, rows) adds nothing (its weight is not read); a
 *   token without any gets zeros.  In fp32 in the order of j, rounded once to Y
 *   [T][M] (yt), overwritten; no overlap.  M any.  T == 0 or M == 0 is an empty call.
 */
ttq_status ttq_moe_combine(const void* R, int rt, int64_t rows, int64_t ldr, const int32_t* pos, const float* w,
                           int64_t T, int64_t topk, int64_t M, void* Y, int yt, int64_t ldy, void* stream);

/*
 * ttq_moe_combine_grad — the gradient of ttq_moe_combine:
 *   dR[pos[t][j]] = w[t][j] dY[t] (rounded to rt; rows that no slot names are
 *   left as they were; no two slots may name one row),
 *   dw[t][j] = sum_o dY[t][o] R[pos[t][j]][o] in fp32 (0 for a slot without a
 *   row), reproducible run to run.
 *   dY: [T][M] (yt), stride lddy; dR: [rows][M] of R's dtype rt, stride lddr,
 *   16-byte aligned, its row stride a multiple of 16 bytes; dw: [T][topk].  dR or
 *   dw may be NULL (R may be, too, without dw).  dR must not overlap R or dY.  M
 *   positive, any.  T == 0 is an empty call.
 */
ttq_status ttq_moe_combine_grad(const void* dY, int yt, int64_t T, int64_t M, int64_t lddy, const void* R, int rt,
                                int64_t rows, int64_t ldr, const int32_t* pos, const float* w, int64_t topk,
                                void* dR, int64_t lddr, float* dw, void* stream);

/* 8-bit weights of E experts of equal shape: codes [E][rows][K] and scale
 * [E][rows], dense, as ttq_quantize_rows writes them for the weight times s;
 * expert e is scaled by s + e * s_stride (s_stride 0: one s for all; else a
 * multiple of 4, at least K). */
typedef struct ttq_expert_i8 {
    const float* s;  int64_t s_stride;
    const int8_t* codes;  const float* scale;
} ttq_expert_i8;

/*
 * ttq_moe_i8 — ttq_moe on 8-bit experts, for long prompts too.
 *   Y[t] = sum_j w[t][j] D_e q(h),  h = act(g) * u / s_down,
 *   [g; u] = G_e q(X[t] / s_in),  e = ids[t][j],
 *   q(.) the row in 8 bits (ttq_quantize_rows), products as in ttq_gemm_i8; h
 *   and the sum over j in fp32, Y rounded once.  ids, w, act, X, Y as for
 *   ttq_moe: a slot whose id is not in [0, E) adds nothing, a token without any
 *   gets zeros, an expert named twice counts twice; an infinite or NaN x / s or
 *   h makes its token's outputs NaN and no other's.  A token's results do not
 *   depend on the other tokens of the call.
 *   K and I multiples of 16, at most 2^17; E <= 1024; 1 <= topk <= 32.  An
 *   expert's gate_up or down codes of 2 GiB or more, T * topk > 2^24 or
 *   T * K >= 2^31 return TTQ_ERR_UNSUPPORTED.  T == 0 or M == 0 is an
 *   empty call.
 *   ws: ttq_moe_i8_workspace_bytes(T, topk, K, I, M, E) bytes, 256-byte aligned;
 *   calls that may run at the same time need workspaces of their own.
 */
typedef struct ttq_moe_i8_args {
    const void* X;  int xt;  int64_t T;  int64_t K;  int64_t ldx;
    const int32_t* ids;  const float* w;  int64_t topk;
    int64_t E;  int64_t I;  int64_t M;
    ttq_expert_i8 gate_up;  ttq_expert_i8 down;
    int act;
    void* Y;  int yt;  int64_t ldy;
} ttq_moe_i8_args;

ttq_status ttq_moe_i8(const ttq_moe_i8_args* args, void* ws, size_t ws_bytes, void* stream);

/* Workspace bytes for ttq_moe_i8 (0 for sizes it does not accept). */
size_t ttq_moe_i8_workspace_bytes(int64_t T, int64_t topk, int64_t K, int64_t I, int64_t M, int64_t E);

/* Static text for a status code. */
const char* ttq_status_str(int status);

/* Text describing the calling thread's last non-OK status ("" if none). */
const char* ttq_last_error(void);

#ifdef __cplusplus
}
#endif

#endif /* TTQ_H */
