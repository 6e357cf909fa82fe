// The mixture-of-experts layer on the matrix cores.
//
// 4-bit codes in groups of 32, 64 or 128 (the sums form): as in the few-token
// projection (qgemv_gs.hip) codes are never expanded to weights: per 32-channel
// subgroup the matrix cores form
//   P[t][o] = sum_j (16 + q_oj) x~_tj,
// slots as the 16 rows and code rows as the 16 columns of a 16x16x32 MFMA,
// and a group adds step P - step (zero + 16) S_t, S_t = sum_j x~_tj, the
// second term as one fp32 16x16x4 MFMA per 128 channels.  16 + q is a bf16
// number whose low byte is 0x80 + 8 q under the high byte 0x41: two bit
// operations and a byte permute per pair of codes; with 16 instead of 128 as
// the offset, the difference of the two terms loses three bits fewer.
// step (zero + 16) is exact in fp32 (11 by 5 bits).
//
// With fp32 X that difference is what rounds most: P is five times as large as
// what it is for, and the outputs were off by 3e-6 to 5e-6 of themselves (2e-7
// to 1e-6 in fp32 arithmetic).  There P is summed over q - c, c the zero as an
// integer, exact in bf16 too; only what is left of a zero, step (c - zero) S_t,
// is added.  Three operations a code instead of two: off by 2e-7 to 3.4e-7; 3 to
// 32 tokens of two of 8 experts, 2048 -> 4096, 42 -> 50, 46 -> 55, 61 -> 75 us; 128
// tokens, 4096 -> 8192, 334 -> 417 us (the weights form below: 6e-7 to 1.4e-6, 61,
// 76, 91 and 639 us).
//
// Other bit widths, and groups of 16 (the weights form): a lane expands the 32
// channels it loads to (code - zero) step, exact in 16 bits and so as two bf16
// terms; about six instructions a code where the sums form takes two.
//
// x~ = x / s (and h for the second product) enters as a sum of NS bf16 terms,
// hi = bf16(x~), then bf16 of what is left: 16 bits for two terms (bf16 X,
// whose own 8 bits one more rounding would nearly double in error), 24 for
// three (fp32 X).  The matrix cores have the room: a step is bound by the
// codes' way from HBM and the integer work of expanding them.  The terms and
// the 16-channel sums are laid out once per row (k_moe_prep; the first
// product's epilogue for h), each 8 channels in the order 0 2 4 6 1 3 5 7
// that the expansion produces, so that a lane loads an operand with one
// 16-byte load.
//
// A wave owns 32 code rows (the first product: 16 gate rows and their 16 up
// rows) and up to 16 slots of one expert; the waves of a workgroup share the
// slots' x~ in LDS, brought there by direct loads, and go through the channels
// in blocks of four chunks of 128, the next block's codes in flight in
// registers while one is multiplied.  With few row groups the blocks of one go
// to several waves, whose tiles are added in wave order through LDS; the second
// product's channels can be split further over workgroups (slices), which the
// sum over a token's slots adds.
//
// What bounds it.  128 tokens, two each of 8 experts, 4096 -> 2 x 14336 -> 4096,
// groups of 64: 443 us, 1.8 TB/s of codes (each read once from memory) and 410
// TFLOP/s counting both terms: vector instructions half of the busy cycles
// (expanding, once per tile of 16 slots), matrix instructions 30%, and waves
// enough to overlap them only with 128 registers each (eight waves instead of
// 16 on a compute unit: 515 us; tiles of 32 slots, which halve the expanding
// but take two operands' registers: 471 us at best).  16 tokens, six each of 64
// experts, 2048 -> 2 x 1056 -> 2048: 78 us, 1.5 slots per tile of 16, where a
// launch per product, its first loads and its end cost as much as the stream.
// (With 128 registers no variant goes to memory for more; some keep up to 20
// scalars in the lanes of a vector register.)
#include "codes.hpp"
#include "common.hpp"
#include "launch.hpp"
#include "lds_dma.hpp"
#include "moe.hpp"

namespace ttq {

constexpr int kMmMaxWaves = 16;
constexpr int kMmRows = 32;                       // code rows per wave
constexpr int kMmChunk = 128;

int64_t moe_pad(int64_t K) { return (K + kMmChunk - 1) / kMmChunk * kMmChunk; }

// ------------------------------------------------------------------ operand layout

constexpr int mm_terms(bool xf32) { return xf32 ? 3 : 2; }

__device__ __forceinline__ u32x4 pack_terms(const float (&x)[8]) {
    // slot order 0 2 4 6 1 3 5 7
    return u32x4{pack_bf16x2(x[0], x[2]), pack_bf16x2(x[4], x[6]), pack_bf16x2(x[1], x[3]), pack_bf16x2(x[5], x[7])};
}
// The bf16 terms of 8 consecutive channels to d, d + kp, ... (elements), and
// their sum as the products see it.
template <int NS>
__device__ __forceinline__ float store_terms(float (&x)[8], uint16_t* d, int64_t kp) {
    float sum = 0.f;
#pragma unroll
    for (int n = 0; n < NS; ++n) {
        const u32x4 v = pack_terms(x);
        *(u32x4*)(d + n * kp) = v;
        const float y[8] = {bf16lo_to_f32(v[0]), bf16lo_to_f32(v[2]), bf16hi_to_f32(v[0]), bf16hi_to_f32(v[2]),
                            bf16lo_to_f32(v[1]), bf16lo_to_f32(v[3]), bf16hi_to_f32(v[1]), bf16hi_to_f32(v[3])};
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            sum += y[e];
            x[e] -= y[e];                         // exact
        }
    }
    return sum;
}

// Block 0 plans (moe.hpp); the others lay out rows of X / s: row r is token
// r (one s for all experts) or slot r (s of the slot's expert; nothing for a
// slot without one).
template <bool XF32>
__global__ __launch_bounds__(kPlanThreads) void k_moe_prep(MoePlan pl, MoePrep a) {
    constexpr int NS = mm_terms(XF32);
    if (blockIdx.x == 0) {
        moe_plan(pl);
        return;
    }
    const int64_t per = a.kp / 8;                 // pieces of 8 channels a row
    const int64_t i = (int64_t)(blockIdx.x - 1) * kPlanThreads + threadIdx.x;
    const int64_t row = i / per, k0 = (i % per) * 8;
    // Rows are whole groups of four threads (kp is a multiple of 128).
    const bool in = row < a.rows;
    int64_t t = row, e = 0;
    bool use = in && k0 < a.K;
    if (a.s_stride != 0 && in) {
        t = row / a.topk;
        e = a.ids[row];
        use = use && e >= 0 && e < a.E;
    }
    float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (use) moe_load_scaled<XF32>(x, a, t, e, k0);
    float sum = 0.f;
    if (in) sum = store_terms<NS>(x, a.xt + row * NS * a.kp + k0, a.kp);
    sum += __shfl_xor(sum, 1);
    if (in && (threadIdx.x & 1) == 0) a.xs[row * (a.kp / 16) + k0 / 16] = sum;
}

// ------------------------------------------------------------------ products

// (x & m) | c in one instruction (the compiler makes two with literals).
__device__ __forceinline__ uint32_t and_or(uint32_t x, uint32_t m, uint32_t c) {
    uint32_t r;
    asm("v_and_or_b32 %0, %1, %2, %3" : "=v"(r) : "v"(x), "s"(m), "v"(c));
    return r;
}

// The bf16 numbers 16 + q of the eight codes of a word, slot order 0 2 4 6 1 3 5 7.
__device__ __forceinline__ u32x4 codes_plus16(uint32_t w) {
    const uint32_t lo = and_or(w << 3, 0x78787878u, 0x80808080u), hi = and_or(w >> 1, 0x78787878u, 0x80808080u);
    constexpr uint32_t k41 = 0x41414141u;
    return u32x4{__builtin_amdgcn_perm(k41, lo, 0x04010400u), __builtin_amdgcn_perm(k41, lo, 0x04030402u),
                 __builtin_amdgcn_perm(k41, hi, 0x04010400u), __builtin_amdgcn_perm(k41, hi, 0x04030402u)};
}

// The bf16 numbers q - z of the eight codes of a word, z an integer of at most
// kMaxShift, slot order as above.
constexpr float kMaxShift = 128.f;
__device__ __forceinline__ u32x4 codes_minus(uint32_t w, float z) {
    const uint32_t lo = w & 0x0F0F0F0Fu, hi = (w >> 4) & 0x0F0F0F0Fu;
    return u32x4{pack_bf16x2(cvt_ubyte<0>(lo) - z, cvt_ubyte<1>(lo) - z), pack_bf16x2(cvt_ubyte<2>(lo) - z, cvt_ubyte<3>(lo) - z),
                 pack_bf16x2(cvt_ubyte<0>(hi) - z, cvt_ubyte<1>(hi) - z), pack_bf16x2(cvt_ubyte<2>(hi) - z, cvt_ubyte<3>(hi) - z)};
}
// The integer that is taken from the codes of a group with this zero (a NaN:
// any; what is left of the zero then is NaN).
__device__ __forceinline__ float shift_of(float zero) { return fminf(fmaxf(rintf(zero), -kMaxShift), kMaxShift); }

constexpr int kMmBlock = 4;                       // chunks whose codes a wave has in flight
// A wave's steps (fp16) and step (zero + 16) (fp32) of a block; or steps with
// what is taken from the codes (pairs of fp16) and what is left of the zeros
// (fp16).
constexpr int kMmStepLds = 3 * 1024;

// LDS of x~: per slot and chunk NS * 256 bytes of terms and 32 of sums, and 32
// a row.  Where the whole slice does not fit,
// half of it holds the chunks being multiplied and half the next ones (kMmMaxX
// bytes, one workgroup of 16 waves on a compute unit); with kMmSmallX bytes
// (two workgroups of eight), for tiles that are mostly expected to fit, all of
// it holds the current ones.
constexpr int mm_unit(int ns) { return ns * 256 + 32; }
constexpr int kMmRowPad = 32;
constexpr int kMmMaxX = 104 * 1024, kMmSmallX = 56 * 1024;
static_assert(kMmMaxX / 2 >= kMmTile * (kMmBlock * mm_unit(3) + kMmRowPad), "a block of every slot's row fits in a half");
static_assert(kMmSmallX >= kMmTile * (kMmBlock * mm_unit(3) + kMmRowPad), "or in all of the small one");
static_assert(kMmMaxX + kMmMaxWaves * kMmStepLds <= 160 * 1024, "LDS of a compute unit");

// GROUP 16, or other codes than 4-bit ones (GROUP then is 16, or 32 for any
// larger one): the weights form (see the head of the file); W2 then is false.
template <int BITS, int GROUP, int NS, bool W2, bool GU>
__global__ __launch_bounds__(kMmMaxWaves * kWave, 4) void k_moe_mfma(MoeMm a) {
    constexpr bool kSums = BITS == 4 && GROUP >= 32;
    constexpr bool kShift = NS == 3;              // sums of q - zero, not 16 + q
    constexpr int NG = kMmChunk / GROUP;          // groups per chunk
    constexpr int SPG = kSums ? GROUP / 32 : 1;   // subgroups per group
    constexpr int SG = GROUP < 32 ? 2 : 1;        // groups of a lane's 32 channels
    constexpr bool kExchange = kSums && GROUP < 128;
    constexpr int D = kSums ? kMmBlock : 2;       // chunks of a block
    constexpr int NB = NG * D;                    // groups per block: 16, 8 or 4
    constexpr int NH = kSums ? (NB > 8 ? 8 : NB) : 4;   // steps a lane loads
    // Loads of a block at least (the compiler may join narrow ones).
    constexpr int kBlockLoads = kSums ? 2 * D + 2 : 2 * D;
    extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
    const MoeTile tl = a.tiles[blockIdx.y];
    if (tl.count == 0) return;
    const int tid = threadIdx.x;
    const int lane = tid & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int nw = blockDim.x / kWave;
    const int nk = a.ksplit, kx = wave % nk;      // this wave's blocks: kx, kx + nk, ...
    const int rw = wave / nk, nr = nw / nk;
    const int r16 = lane & 15, q = lane >> 4;
    const int64_t K = a.K, R = GU ? 2 * a.rows : a.rows;
    const int64_t wpr = K * BITS / 32, gpr = K / (kSums ? GROUP : a.group);
    const int64_t o0 = ((int64_t)blockIdx.x * nr + rw) * (GU ? kMmRows / 2 : kMmRows);
    const rsrc_t rc = make_rsrc(a.codes + (int64_t)tl.expert * R * wpr, R * wpr * 4);
    uint32_t sa, za;
    const rsrc_t rsc = moe_half_rsrc(a.scale + (int64_t)tl.expert * R * gpr, R * gpr * 2, sa);
    const rsrc_t rze = moe_half_rsrc(a.zero + (int64_t)tl.expert * R * gpr, R * gpr * 2, za);
    // Code row of column r of column tile rt; rows past the end are clamped
    // and their outputs not used.
    auto row_of = [&](int rt, int r) -> int64_t {
        if constexpr (GU) return min(o0 + r, a.rows - 1) + (rt ? a.rows : 0);
        else return min(o0 + 16 * rt + r, a.rows - 1);
    };
    const uint32_t co[2] = {(uint32_t)(row_of(0, r16) * wpr * 4 + 4 * BITS * q),
                            (uint32_t)(row_of(1, r16) * wpr * 4 + 4 * BITS * q)};
    const uint32_t wo[2] = {(uint32_t)(row_of(0, r16) * gpr * 2), (uint32_t)(row_of(1, r16) * gpr * 2)};   // weights form
    // Steps and zeros of a block: lane (row, part) of the 32 rows.
    constexpr int kParts = kSums ? NB / NH : 1;
    const int grow = lane / kParts & 31, gpart = lane % kParts;
    const uint32_t go = (uint32_t)((row_of(grow >> 4, grow & 15) * gpr + gpart * NH) * 2);
    const int nch = (int)(a.kp / kMmChunk);
    const int cb = (int)blockIdx.z * a.per_slice;
    const int cnt = min(nch, cb + a.per_slice) - cb;   // chunks of this slice

    // x~ and its sums of kb chunks at a time.
    constexpr int kUnit = mm_unit(NS);
    const int rows = tl.count;
    const int xrow = a.order[tl.first + min(lane & 15, rows - 1)] / a.div;   // operand row of slot lane % 16
    int kb = (cnt + D - 1) & ~(D - 1), half = 0;
    if (rows * (kb * kUnit + kMmRowPad) > a.xbytes) {
        half = a.xbytes > kMmSmallX ? a.xbytes / 2 & ~255 : 0;
        kb = ((half ? half : a.xbytes) / rows - kMmRowPad) / kUnit & ~(D - 1);
    }
    const int rowb = NS * kb * 256, srowb = kb * 32 + 16;
    unsigned char* const xb = smem + nw * kMmStepLds;
    // Straight from memory into LDS: a wave's instruction takes four pairs of
    // chunk and term (256 bytes each, terms next to each other) of one row, or
    // a row's sums.  Row r has its 16-byte pieces at their place exclusive-or'ed
    // with f(r), so that the 16 rows of a fragment lie in different banks, also
    // where the hardware pairs rows of one quarter with others of the next (f:
    // r, or with the quarters 64 bytes apart its bit pairs swapped).
    auto swizzle = [](int r) __attribute__((always_inline)) { return kExchange ? r : (r & 3) << 2 | r >> 2; };
    auto stage = [&](int i0, unsigned char* to) __attribute__((always_inline)) {
        const int units = NS * kb, per = (units + 3) / 4 + 1;
        for (int u = wave; u < rows * per; u += nw) {
            const int r = u / per, w = u - r * per;
            const int64_t xr = __builtin_amdgcn_readlane(xrow, r);
            if (w == per - 1) {
                const rsrc_t rs = make_rsrc(a.xs + xr * (a.kp / 16), a.kp / 4);
                for (int h = 0; h * 32 < kb; ++h)
                    if (lane < 2 * (kb - 32 * h))
                        dma_to_lds<16>(rs, to + rows * rowb + r * srowb + h * 1024, lane * 16, (cb + i0 + 32 * h) * 32);
            } else {
                const rsrc_t rx = make_rsrc(a.xt + xr * NS * a.kp, NS * a.kp * 2);
                const int v = 4 * w + q, c = v / NS, n = v - c * NS;
                if (v < units)
                    dma_to_lds<16>(rx, to + r * rowb + w * 1024,
                                   (int)(n * a.kp * 2) + c * 256 + ((r16 ^ swizzle(r)) * 16), (cb + i0) * 256);
            }
        }
    };
    stage(0, xb);

    // Codes, steps and zeros of a block; chunks past the slice are asked for
    // behind the buffer (zeros, no traffic), so that a block always has its
    // loads and the waits below can count them.
    struct Code {
        CodeWords<BITS> c;
        uint16_t st[kSums ? 1 : SG], ze[kSums ? 1 : SG];   // weights form: of the lane's 32 channels
    };
    Code ring[D][2];
    uint32_t sw[NH / 2], zw[NH / 2];
    // Ordinary loads: a line of a row serves two chunks, and the tiles of one
    // expert read the same codes (128 tokens over 8 experts: 557 us against 616
    // with streaming ones).
    auto load = [&](int u, int i) __attribute__((always_inline)) {
        const uint32_t at = i < cnt ? (uint32_t)(cb + i) * (16 * BITS) : 0x80000000u;
#pragma unroll
        for (int rt = 0; rt < 2; ++rt) {
            Code& c = ring[u][rt];
            const int off = (int)(co[rt] + at);
            if constexpr (BITS >= 4) {
                const u32x4 v = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rc, off, 0, 0));
#pragma unroll
                for (int w = 0; w < 4; ++w) c.c.w[w] = v[w];
                if constexpr (BITS == 5) c.c.w[4] = __builtin_amdgcn_raw_buffer_load_b32(rc, off + 16, 0, 0);
            } else if constexpr (BITS == 3) {
                const auto v = __builtin_amdgcn_raw_buffer_load_b96(rc, off, 0, 0);
#pragma unroll
                for (int w = 0; w < 3; ++w) c.c.w[w] = v[w];
            } else {
                const u32x2 v = __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(rc, off, 0, 0));
                c.c.w[0] = v[0];
                c.c.w[1] = v[1];
            }
            if constexpr (!kSums) {
                const int ch = (cb + i) * kMmChunk + 32 * q;   // first channel of this lane
                const uint32_t g = i < cnt && ch < K ? wo[rt] + (uint32_t)(SG == 2 ? ch / 16 : ch / a.group) * 2 : 0x80000000u;
#pragma unroll
                for (int h = 0; h < SG; ++h) {
                    c.st[h] = __builtin_amdgcn_raw_buffer_load_b16(rsc, (int)(g + sa + 2 * h), 0, 0);
                    c.ze[h] = __builtin_amdgcn_raw_buffer_load_b16(rze, (int)(g + za + 2 * h), 0, 0);
                }
            }
        }
    };
    auto load_sz = [&](int i) __attribute__((always_inline)) {
        if constexpr (kSums) {
            const uint32_t off = go + (i < cnt ? (uint32_t)(cb + i) * (NG * 2) : 0x80000000u);
            moe_load_halves<NH, W2>(sw, rsc, off + sa);
            moe_load_halves<NH, W2>(zw, rze, off + za);
        }
    };
    int b = D * kx;                               // first chunk of the block
    __builtin_amdgcn_sched_barrier(0);
    load_sz(b);
#pragma unroll
    for (int u = 0; u < D; ++u) load(u, b + u);
    __builtin_amdgcn_sched_barrier(0);

    // Lanes past the tile's slots repeat its first one; their outputs are not
    // used.  In quarter q, MFMA j takes channels 32 j + 8 q ..+7 of the chunk
    // (the codes after the exchange of quarters), with one group per chunk or
    // weights 32 q + 8 j ..+7 (no exchange needed).
    const int rl = r16 < rows ? r16 : 0;
    uint32_t xo[4];                               // bytes from the buffer's start, of MFMA j's piece
#pragma unroll
    for (int j = 0; j < 4; ++j) xo[j] = rl * rowb + (((kExchange ? 4 * j + q : 4 * q + j) ^ swizzle(rl)) * 16);
    const uint32_t so = rows * rowb + rl * srowb + 8 * q;
    unsigned char* const my = smem + wave * kMmStepLds;
    uint16_t* const st_l = (uint16_t*)my;         // [32][NB]
    float* const nb_l = (float*)(my + 1024);      // [32][NB]
    uint32_t* const sz_l = (uint32_t*)my;         // kShift: [32][NB]
    uint16_t* const rest_l = (uint16_t*)(my + 2048);
    const int gq = NG == 4 ? q : NG == 2 ? q >> 1 : 0;   // group of subgroup q within a chunk

    f32x4 acc[2] = {f32x4{0.f, 0.f, 0.f, 0.f}, f32x4{0.f, 0.f, 0.f, 0.f}};
    auto multiply_weights = [&](int u, const uint32_t (&xa)[4]) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            u32x4 wt[2][2];                       // the weights' terms, slot order 0 2 4 6 1 3 5 7
#pragma unroll
            for (int rt = 0; rt < 2; ++rt) {
                const Code& c = ring[u][rt];
                const float st = f16_to_f32(c.st[8 * j / 16 % SG]), nz = -f16_to_f32(c.ze[8 * j / 16 % SG]) * st;
                float w[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) w[e] = __builtin_fmaf((float)code_at<BITS>(c.c, 8 * j + e), st, nz);
                wt[rt][0] = pack_terms(w);
#pragma unroll
                for (int e = 0; e < 4; ++e) {     // element e: channels kLo[e] and kLo[e] + 2
                    constexpr int kLo[4] = {0, 4, 1, 5};
                    w[kLo[e]] -= bf16lo_to_f32(wt[rt][0][e]);
                    w[kLo[e] + 2] -= bf16hi_to_f32(wt[rt][0][e]);
                }
                wt[rt][1] = pack_terms(w);
            }
#pragma unroll
            for (int n = NS - 1; n >= 0; --n) {
                const u32x4 x = *(const u32x4*)(smem + xa[j] + (u * NS + n) * 256);
#pragma unroll
                for (int h = 1; h >= 0; --h)
#pragma unroll
                    for (int rt = 0; rt < 2; ++rt) acc[rt] = mfma_16x16x32(x, wt[rt][h], acc[rt]);
            }
        }
    };
    // xa, sa: the block's operand and sums in LDS.
    auto multiply = [&](int u, const uint32_t (&xa)[4], uint32_t sa) __attribute__((always_inline)) {
        if constexpr (!kSums) {
            multiply_weights(u, xa);
            return;
        }
        const float* sp = (const float*)(smem + sa + 32 * u);
        const float si = sp[0] + sp[1];
        f32x4 p[2];
        u32x4 w4[2];
        uint32_t st[2][(NG + 1) / 2];             // steps
        float nb[2];                              // the zero terms' factors: -step (zero + 16), or what is left of it
        uint32_t sz[2][kShift ? NG : 1];
#pragma unroll
        for (int rt = 0; rt < 2; ++rt) {
            w4[rt] = u32x4{ring[u][rt].c.w[0], ring[u][rt].c.w[1], ring[u][rt].c.w[2], ring[u][rt].c.w[BITS > 3 ? 3 : 0]};
            if constexpr (kExchange) swap_quarters(w4[rt]);
            p[rt] = f32x4{0.f, 0.f, 0.f, 0.f};
            const int g = (16 * rt + r16) * NB + u * NG;
            if constexpr (kShift) {
#pragma unroll
                for (int v = 0; v < NG; ++v) sz[rt][v] = sz_l[g + v];
                nb[rt] = half_at(sz_l[g + gq], false) * f16_to_f32(rest_l[g + gq]);
            } else {
                if constexpr (NG == 1) st[rt][0] = st_l[g];
                else
#pragma unroll
                    for (int v = 0; v < NG / 2; ++v) st[rt][v] = ((const uint32_t*)(st_l + g))[v];
                nb[rt] = nb_l[g + gq];
            }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            u32x4 bb[2];
#pragma unroll
            for (int rt = 0; rt < 2; ++rt) {
                if constexpr (kShift) bb[rt] = codes_minus(w4[rt][j], half_at(sz[rt][j / SPG], true));
                else bb[rt] = codes_plus16(w4[rt][j]);
            }
#pragma unroll
            for (int n = NS - 1; n >= 0; --n) {
                const u32x4 x = *(const u32x4*)(smem + xa[j] + (u * NS + n) * 256);
#pragma unroll
                for (int rt = 0; rt < 2; ++rt) p[rt] = mfma_16x16x32(x, bb[rt], p[rt]);
            }
            if ((j + 1) % SPG == 0) {
                const int g = j / SPG;
#pragma unroll
                for (int rt = 0; rt < 2; ++rt) {
                    float s;
                    if constexpr (kShift) s = half_at(sz[rt][g], false);
                    else s = half_at(st[rt][g / 2], g & 1);
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[rt][e] = __builtin_fmaf(s, p[rt][e], acc[rt][e]);
                    p[rt] = f32x4{0.f, 0.f, 0.f, 0.f};
                }
            }
        }
#pragma unroll
        for (int rt = 0; rt < 2; ++rt) acc[rt] = __builtin_amdgcn_mfma_f32_16x16x4f32(si, nb[rt], acc[rt], 0, 0, 0);
    };
    // Everything but this block's loads has arrived: x~ has.
    wait_vmcnt<kBlockLoads>();
    unsigned char *x0 = xb, *x1 = xb + half;
    for (int i0 = 0; i0 < cnt; i0 += kb) {
        sync_lds();                               // every wave's part of x~; the half multiplied last is free
        if (half == 0 && i0 > 0) {                // one buffer: refilled between two barriers
            stage(i0, x0);
            wait_vmcnt<0>();
            sync_lds();
        }
        const int e = min(cnt, i0 + kb);
        if (half != 0 && e < cnt) stage(e, x1);
        bool newer = false;                       // loads were issued after the stage's
        for (; b < e; b += D * nk) {
            // This block's steps into the wave's part of LDS (its reads of the
            // block before are done: LDS operations of a wave keep their order).
            if (kSums && lane < 32 * kParts) {
                const int left = (int)gpr - (cb + b) * NG - gpart * NH;   // groups of the row from here
                if (left < NH)                    // behind the row: the next row's, which may be anything
#pragma unroll
                    for (int v = 0; v < NH; ++v)
                        if (v >= left) {
                            sw[v / 2] &= v & 1 ? 0xFFFFu : 0u;
                            zw[v / 2] &= v & 1 ? 0xFFFFu : 0u;
                        }
                if constexpr (kShift) {
#pragma unroll
                    for (int v = 0; v < NH; ++v) {
                        const float z = half_at(zw[v / 2], v & 1), c = shift_of(z);
                        const uint32_t st = v & 1 ? sw[v / 2] >> 16 : sw[v / 2] & 0xFFFFu;
                        sz_l[grow * NB + gpart * NH + v] = st | (uint32_t)f32_to_f16_rne(c) << 16;
                        rest_l[grow * NB + gpart * NH + v] = f32_to_f16_rne(c - z);   // exact
                    }
                } else {
#pragma unroll
                    for (int v = 0; v < NH / 2; ++v) ((uint32_t*)(st_l + grow * NB + gpart * NH))[v] = sw[v];
#pragma unroll
                    for (int v = 0; v < NH; ++v)
                        nb_l[grow * NB + gpart * NH + v] = -(half_at(sw[v / 2], v & 1) * (half_at(zw[v / 2], v & 1) + 16.f));
                }
            }
            __builtin_amdgcn_wave_barrier();
            const int bn = b + D * nk;
            load_sz(bn);
            uint32_t xa[4];
            const uint32_t x00 = (uint32_t)(x0 - smem);
#pragma unroll
            for (int j = 0; j < 4; ++j) xa[j] = xo[j] + (x00 + (b - i0) * (NS * 256));
            const uint32_t xsum = so + (x00 + (b - i0) * 32);
#pragma unroll
            for (int u = 0; u < D; ++u) {
                if (b + u < e) multiply(u, xa, xsum);
                load(u, bn + u);
                __builtin_amdgcn_sched_barrier(0);
            }
            newer = true;
        }
        if (half != 0 && e < cnt) {               // uniform
            if (newer) wait_vmcnt<kBlockLoads>();
            else wait_vmcnt<0>();
        }
        unsigned char* t = x0;
        x0 = x1;
        x1 = t;
    }
    if (nk > 1) {                                 // uniform: the waves of a row group added in order
        sync_lds();                               // x~ has been read
        f32x4* red = (f32x4*)xb;
#pragma unroll
        for (int rt = 0; rt < 2; ++rt) red[(wave * 2 + rt) * kWave + lane] = acc[rt];
        sync_lds();
        if (kx == 0)
            for (int w = 1; w < nk; ++w)
#pragma unroll
                for (int rt = 0; rt < 2; ++rt) {
                    const f32x4 v = red[((wave + w) * 2 + rt) * kWave + lane];
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[rt][e] += v[e];
                }
    }
    if (kx != 0) return;

    // Lane: slots 4 q + e of row r16 of each column tile.
    if constexpr (!GU) {
#pragma unroll
        for (int rt = 0; rt < 2; ++rt) {
            const int64_t o = o0 + 16 * rt + r16;
            if (o < a.rows) {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (4 * q + e < rows)
                        a.p[((int64_t)blockIdx.z * a.slots + a.order[tl.first + 4 * q + e]) * a.ldp + o] = acc[rt][e];
            }
        }
    } else {
        // h = act(g) u w / s_down of 4 slots and one channel; through the
        // wave's part of LDS to the second product's operand: lane (slot, 8
        // channels).
        const int64_t o = o0 + r16;
        f32x4 h;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int t = 4 * q + e;
            h[e] = 0.f;
            if (o < a.rows && t < rows) {
                const float f = a.w[a.order[tl.first + t]] / a.s_out[tl.expert * a.s_out_stride + o];
                h[e] = moe_act(acc[0][e], a.act) * acc[1][e] * f;
            }
        }
        f32x4* hb = (f32x4*)my;
        __builtin_amdgcn_wave_barrier();
        hb[lane] = h;
        __builtin_amdgcn_wave_barrier();
        const int t = (lane >> 1) & 15, c8 = lane & 1;
        float x[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = ((const float*)&hb[16 * (t >> 2) + 8 * c8 + e])[t & 3];
        const bool in = lane < 32 && t < rows && o0 < a.hp;
        const int64_t hs = a.order[tl.first + (in ? t : 0)];
        float s = 0.f;
        if (in) s = store_terms<NS>(x, a.ht + hs * NS * a.hp + o0 + 8 * c8, a.hp);
        s += __shfl_xor(s, 1);
        if (in && c8 == 0) a.hs[hs * (a.hp / 16) + o0 / 16] = s;
    }
}

// ------------------------------------------------------------------ host

// Waves of a workgroup: row groups of 32 code rows (they share x~ in LDS).
// Eight, two workgroups on a compute unit, where the operands fit or the
// experts have at most four slots on average (their tiles mostly fit); else
// 16 with two buffers (measured, 128 tokens over 8 experts, 32 slots each: 633
// us against 661 with eight waves and one buffer; 16 tokens over 64 experts,
// 1.5 slots each: 97 us against 87; both before the steps that followed).
// Where there are fewer than three waves per SIMD, the blocks of a row group's
// channels go to up to four waves, and where the chip would not get its
// workgroups, they are smaller.
struct MmShape {
    int nr, nk, xbytes;
    size_t lds() const { return (size_t)nr * nk * kMmStepLds + xbytes; }
};
static MmShape mm_shape(int64_t waves, int64_t tiles, int64_t chunks, int64_t n, int64_t E, int ns) {
    MmShape s{0, 1, 0};
    const int64_t rows = n < kMmTile ? n : kMmTile, c4 = (chunks + kMmBlock - 1) / kMmBlock * kMmBlock;
    const int64_t need = rows * (c4 * mm_unit(ns) + kMmRowPad);
    const bool wide = need > kMmSmallX && n > 4 * E;
    const int64_t most_x = wide ? kMmMaxX : kMmSmallX;
    s.xbytes = (int)(need < most_x ? (need + 15) / 16 * 16 : most_x);
    const int most = wide ? 16 : 8;
    const int64_t wgs = wide ? 256 : 512;
    while (s.nk < 4 && waves * tiles * s.nk < 3 * kSimds && chunks >= 2 * kMmBlock * s.nk) s.nk *= 2;
    s.nr = most / s.nk;
    while (s.nr > 1 && s.nr * s.nk > 2 && (waves + s.nr - 1) / s.nr * tiles < wgs) s.nr /= 2;
    const int red = s.nr * s.nk * 2 * kWave * 16;   // the waves' tiles, where they are added
    if (s.nk > 1 && s.xbytes < red) s.xbytes = red;
    return s;
}

// Slices of the second product's channels: enough waves to fill the chip, at
// least eight chunks each.
int moe_slices(int64_t n, int64_t E, int64_t I, int64_t M) {
    const int64_t tiles = moe_tiles(n, E, kMmTile), waves = (M + kMmRows - 1) / kMmRows * tiles;
    if (waves == 0) return 1;                     // an empty call
    const int64_t chunks = moe_pad(I) / kMmChunk, most = chunks / 8 > 0 ? chunks / 8 : 1;
    // The wide workgroups (one of 16 waves on a compute unit, for experts of
    // more than four slots) come in several rounds: 128 tokens over 8 experts,
    // 14336 -> 4096, 556 us with one slice (160 workgroups), 441 us with three.
    const int64_t want = n > 4 * E ? 6144 : 2048;
    int64_t s = (want + waves - 1) / waves;
    if (s > most) s = most;
    return (int)(s < 1 ? 1 : s > 16 ? 16 : s);
}

template <int NS, bool GU>
static hipError_t launch_mm(const MoeMm& p, int bits, int group, dim3 grid, int waves, size_t lds, hipStream_t st) {
    const bool w2 = moe_w2(p.scale, p.zero, p.K / group);
#define TTQ_MW(B, G) \
    return launch_kernel(k_moe_mfma<B, G, NS, false, GU>, grid, dim3(waves * kWave), lds, st, nullptr, nullptr, p)
    if (bits == 4 && group == 16) TTQ_MW(4, 16);
    if (bits != 4) {
        if (group == 16) {
            if (bits == 2) TTQ_MW(2, 16);
            if (bits == 3) TTQ_MW(3, 16);
            TTQ_MW(5, 16);
        }
        if (bits == 2) TTQ_MW(2, 32);
        if (bits == 3) TTQ_MW(3, 32);
        TTQ_MW(5, 32);
    }
#undef TTQ_MW
#define TTQ_MM(G)                                                                                                     \
    return w2 ? launch_kernel(k_moe_mfma<4, G, NS, true, GU>, grid, dim3(waves * kWave), lds, st, nullptr, nullptr, p)   \
              : launch_kernel(k_moe_mfma<4, G, NS, false, GU>, grid, dim3(waves * kWave), lds, st, nullptr, nullptr, p)
    switch (group) {
        case 32: TTQ_MM(32);
        case 64: TTQ_MM(64);
        case 128: TTQ_MM(128);
    }
#undef TTQ_MM
    return hipErrorInvalidValue;
}

// Chunks of a slice where `sl` are wanted.  An even number: a slice's first step
// lies at a word's start also where a chunk is one group (a load at half a word
// would lose the steps of the last row's end, cut off there by the buffer's
// word-wise bound).
static int mm_per_slice(int64_t chunks, int64_t sl) { return (int)((chunks + sl - 1) / sl + 1) & ~1; }

// d.p = the products of n operand rows and d.rows code rows, in slices of
// per_slice chunks.
template <int NS>
static hipError_t launch_rows(MoeMm d, int bits, int64_t nt, int64_t n, int64_t E, int per_slice, hipStream_t st) {
    const int64_t chunks = d.kp / kMmChunk, nsl = (chunks + per_slice - 1) / per_slice;
    const int64_t dw = (d.rows + kMmRows - 1) / kMmRows;
    const MmShape v = mm_shape(dw, nt * nsl, per_slice, n, E, NS);
    d.per_slice = per_slice; d.ksplit = v.nk; d.xbytes = v.xbytes;
    return launch_mm<NS, false>(d, bits, d.group, dim3((unsigned)((dw + v.nr - 1) / v.nr), (unsigned)nt, (unsigned)nsl),
                                v.nr * v.nk, v.lds(), st);
}

template <bool XF32>
static hipError_t launch_layer(const ttq_moe_args* a, const MoeLayout& L, char* ws, hipStream_t st) {
    constexpr int NS = mm_terms(XF32);
    const int64_t n = a->T * a->topk, kp = moe_pad(a->K), ip = moe_pad(a->I);
    const int64_t nt = moe_tiles(n, a->E, kMmTile);
    MoePlan pl{a->ids, (int)n, (int)a->E, kMmTile, (int)nt, (int32_t*)(ws + L.order), (MoeTile*)(ws + L.tiles)};
    MoePrep pr = moe_prep_of(a, kp);
    pr.xt = (uint16_t*)(ws + L.xt); pr.xs = (float*)(ws + L.xs);
    const dim3 pg((unsigned)(1 + (pr.rows * (kp / 8) + kPlanThreads - 1) / kPlanThreads));
    if (hipError_t e = launch_kernel(k_moe_prep<XF32>, pg, dim3(kPlanThreads), 0, st, nullptr, nullptr, pl, pr))
        return e;
    MoeMm p{};
    p.tiles = pl.tiles; p.order = pl.order; p.slots = n;
    p.xt = pr.xt; p.xs = pr.xs; p.K = a->K; p.group = a->group; p.kp = kp; p.rows = a->I; p.div = pr.s_stride ? 1 : (int)a->topk;
    p.codes = (const uint32_t*)a->gate_up.codes; p.scale = a->gate_up.scale_f16; p.zero = a->gate_up.zero_f16;
    p.per_slice = (int)(kp / kMmChunk);
    p.w = a->w; p.s_out = a->down.s; p.s_out_stride = a->down.s_stride; p.act = a->act;
    p.ht = (uint16_t*)(ws + L.h); p.hs = (float*)(ws + L.hs); p.hp = ip;
    const int64_t gw = ip / 16;
    const MmShape g = mm_shape(gw, nt, p.per_slice, n, a->E, NS);
    p.ksplit = g.nk; p.xbytes = g.xbytes;
    if (hipError_t e = launch_mm<NS, true>(p, a->bits, a->group, dim3((unsigned)((gw + g.nr - 1) / g.nr), (unsigned)nt),
                                           g.nr * g.nk, g.lds(), st))
        return e;
    MoeMm d{};
    d.tiles = pl.tiles; d.order = pl.order; d.slots = n;
    d.xt = p.ht; d.xs = p.hs; d.K = a->I; d.group = a->group; d.kp = ip; d.rows = a->M; d.div = 1;
    d.codes = (const uint32_t*)a->down.codes; d.scale = a->down.scale_f16; d.zero = a->down.zero_f16;
    d.p = (float*)(ws + L.p); d.ldp = a->M;
    const int64_t chunks = ip / kMmChunk;
    const int per = mm_per_slice(chunks, moe_slices(n, a->E, a->I, a->M));
    if (hipError_t e = launch_rows<NS>(d, a->bits, nt, n, a->E, per, st)) return e;
    return launch_moe_sum(a, d.p, (int)((chunks + per - 1) / per), st);
}

hipError_t launch_moe_mfma(const ttq_moe_args* a, const MoeLayout& L, char* ws, hipStream_t st) {
    return a->xt == TTQ_F32 ? launch_layer<true>(a, L, ws, st) : launch_layer<false>(a, L, ws, st);
}

// ------------------------------------------------------------------ one weight for all tokens

// A projection of fp32 X with x / s to 24 bits: one expert's product, off by
// 1.5e-7 to 3.4e-7 of the outputs (two bf16 halves of x and of the weight: 3e-6).
// In ttq_qgemm_adapters, 4096 -> 4096, 4-bit groups of 32 (in brackets with the
// halves' kernels): 16 tokens 29 (30) us, 64 47 (60), 300 114 (333), 1024 233 (355);
// 16 tokens 2048 -> 2048, where one launch more counts, 31 (21).  At most
// kProjTokens tokens a pass, and of code rows what a buffer descriptor holds.
constexpr int64_t kProjTokens = 4096;

struct ProjLayout {
    size_t p, order, tiles, xt, xs, total;
};
static ProjLayout proj_layout(int64_t T, int64_t K, int64_t M) {
    auto up = [](size_t n) { return (n + 255) / 256 * 256; };
    const int64_t n = T < kProjTokens ? T : kProjTokens, kp = moe_pad(K);
    ProjLayout L{};
    L.p = 0;
    L.order = L.p + up((size_t)proj_f32_parts(T, K, M) * T * M * 4);
    L.tiles = L.order + up((size_t)n * 4);
    L.xt = L.tiles + up((size_t)moe_tiles(n, 1, kMmTile) * sizeof(MoeTile));
    L.xs = L.xt + up((size_t)n * mm_terms(true) * kp * 2);
    L.total = L.xs + up((size_t)n * (kp / 16) * 4);
    return L;
}
static int proj_per_slice(int64_t T, int64_t K, int64_t M) {
    return mm_per_slice(moe_pad(K) / kMmChunk, moe_slices(T < kProjTokens ? T : kProjTokens, 1, K, M));
}
int proj_f32_parts(int64_t T, int64_t K, int64_t M) {
    const int per = proj_per_slice(T, K, M);
    return (int)((moe_pad(K) / kMmChunk + per - 1) / per);
}
size_t proj_f32_ws_bytes(int64_t T, int64_t K, int64_t M) { return proj_layout(T, K, M).total; }

hipError_t launch_proj_f32(const float* X, int64_t T, int64_t K, int64_t ldx, const float* s, const uint32_t* codes,
                           const uint16_t* scale, const uint16_t* zero, int64_t M, int bits, int group, char* ws,
                           hipStream_t st) {
    constexpr int NS = mm_terms(true);
    const ProjLayout L = proj_layout(T, K, M);
    const int64_t kp = moe_pad(K), wpr = K * bits / 32;
    const int64_t most = (((int64_t)1 << 31) - 1) / (wpr * 4) / kMmRows * kMmRows;   // code rows
    for (int64_t t0 = 0; t0 < T; t0 += kProjTokens) {
        const int64_t n = T - t0 < kProjTokens ? T - t0 : kProjTokens, nt = moe_tiles(n, 1, kMmTile);
        MoePlan pl{nullptr, (int)n, 1, kMmTile, (int)nt, (int32_t*)(ws + L.order), (MoeTile*)(ws + L.tiles)};
        MoePrep pr{};
        pr.X = X + t0 * ldx; pr.ldx = ldx; pr.K = K; pr.kp = kp; pr.rows = n; pr.s = s;
        pr.xt = (uint16_t*)(ws + L.xt); pr.xs = (float*)(ws + L.xs);
        const dim3 pg((unsigned)(1 + (n * (kp / 8) + kPlanThreads - 1) / kPlanThreads));
        if (hipError_t e = launch_kernel(k_moe_prep<true>, pg, dim3(kPlanThreads), 0, st, nullptr, nullptr, pl, pr)) return e;
        for (int64_t r0 = 0; r0 < M; r0 += most) {
            MoeMm d{};
            d.tiles = pl.tiles; d.order = pl.order; d.slots = T;
            d.xt = pr.xt; d.xs = pr.xs; d.K = K; d.group = group; d.kp = kp; d.div = 1;
            d.rows = M - r0 < most ? M - r0 : most;
            d.codes = codes + r0 * wpr; d.scale = scale + r0 * (K / group); d.zero = zero + r0 * (K / group);
            d.p = (float*)(ws + L.p) + t0 * M + r0; d.ldp = M;
            if (hipError_t e = launch_rows<NS>(d, bits, nt, n, 1, proj_per_slice(T, K, M), st)) return e;
        }
    }
    return hipSuccess;
}

}  // namespace ttq
