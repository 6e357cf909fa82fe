// The mixture-of-experts layer for one or two slots an expert (4-bit codes,
// groups of 32, 64 or 128): 4-bit integer dot products.
//
// With so few rows a matrix-core tile is mostly empty, and expanding the
// codes for it costs more than the products; here they are multiplied as they
// lie in memory.  x~ (x / s, or h) is held per 32 channels as integers X of ND
// base-16 digits times a scale: x~_j = sx X_j, |X_j| <= 7 (16^ND - 1) / 15,
// off by at most half of sx, i.e. 2^-19 (five digits, bf16 X) or 2^-23 (six,
// fp32 X) of the largest of the 32.  Digits lie in [-8, 7], one nibble each,
// in the order of the codes, and q ^ 8 is q - 8 as a nibble, so eight products
// are one v_dot8_i32_i4:
//   sum_j (q_j - zero) x~_j = sx (sum_d 16^d dot(q - 8, X_d) + (8 - zero) sum_j X_j),
// the integers exact, the rest fp32.  Per 32 codes and slot: 4 ND dots and
// about ten more instructions, half of the matrix-core form's at one slot.
//
// A wave owns 64 code rows (the first product: 32 gate rows and their 32 up
// rows); a load takes 512 channels of four rows, 256 consecutive bytes each
// (the matrix cores' fragments, 16 rows x 64 bytes, read the same codes a
// fifth slower).  A piece is 512 channels: lane (g, f) holds field f of 32
// channels, rows 4 r + g in step r; steps and zeros of a piece come row by row
// in 16-byte loads and pass through LDS.  Sums over the 16 fields by a fixed
// exchange, over the waves of a row group (each its own pieces) in order
// through LDS.
#include "common.hpp"
#include "launch.hpp"
#include "lds_dma.hpp"
#include "moe.hpp"

namespace ttq {

constexpr int kMdMaxWaves = 8;
constexpr int kMdRows = 64;                       // code rows per wave
constexpr int kMdPiece = 512;
constexpr int kMdRing = 8;                        // code loads in flight

int64_t moe_dot_pad(int64_t K) { return (K + kMdPiece - 1) / kMdPiece * kMdPiece; }

constexpr int md_digits(bool xf32) { return xf32 ? 6 : 5; }

template <int ND>
struct Digits {
    static constexpr int kMax = 7 * ((1 << (4 * ND)) - 1) / 15;   // the largest number of ND digits <= 7
    static constexpr uint32_t kBias = 0x88888888u >> (32 - 4 * ND);
};
// u = X + 88..8 has the digits plus 8 as nibbles; nibble d of it as a signed digit.
__device__ __forceinline__ uint32_t digit_of(uint32_t u, int d) { return ((u >> (4 * d)) & 15u) ^ 8u; }

// |x| as bits, whose largest is a NaN's if there is one (fmax would drop it).
__device__ __forceinline__ uint32_t abs_bits(float x) { return __builtin_bit_cast(uint32_t, x) & 0x7FFFFFFFu; }
// x as an integer of ND digits where the largest of its 32 is mx: by up * inv,
// `up` so that kMax / mx stays finite.  Of no meaning (but defined) where mx is
// no finite number: the scale is NaN then.
template <int ND>
struct ToDigits {
    float up, inv;
    __device__ __forceinline__ explicit ToDigits(float mx) {
        up = mx < 0x1p-64f ? 0x1p64f : 1.f;
        inv = mx > 0.f ? (float)Digits<ND>::kMax / (mx * up) : 0.f;
    }
    __device__ __forceinline__ int operator()(float x) const {
        constexpr float m = (float)Digits<ND>::kMax;
        return (int)rintf(fminf(fmaxf(x * up * inv, -m), m));
    }
};

// The scale of 32 channels.  An infinite one would give signed infinities
// (and the digits of an infinity have no sign), so it is NaN as well.
template <int ND>
__device__ __forceinline__ float digit_scale(float mx) {
    return mx < __builtin_inff() ? mx / (float)Digits<ND>::kMax : __builtin_nanf("");
}

// x~ of a row: digits [ND][kp / 8] words, then per 32 channels the scale and
// the sum of the integers, [2][kp / 32] floats.
template <int ND>
__device__ __forceinline__ int64_t digit_row_words(int64_t kp) { return ND * (kp / 8) + 2 * (kp / 32); }

// ------------------------------------------------------------------ operand

// Block 0 plans; the others lay out X / s per slot: a thread has 8 channels.
template <bool XF32>
__global__ __launch_bounds__(kPlanThreads) void k_moe_dot_prep(MoePlan pl, MoePrep a, uint32_t* __restrict__ out) {
    constexpr int ND = md_digits(XF32);
    if (blockIdx.x == 0) {
        moe_plan(pl);
        return;
    }
    const int64_t per = a.kp / 8;
    const int64_t i = (int64_t)(blockIdx.x - 1) * kPlanThreads + threadIdx.x;
    const int64_t row = i / per, k8 = i % per, k0 = k8 * 8;
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
    uint32_t mb = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) mb = max(mb, abs_bits(x[j]));
    mb = max(mb, (uint32_t)__shfl_xor((int)mb, 1));
    mb = max(mb, (uint32_t)__shfl_xor((int)mb, 2));
    const float mx = __builtin_bit_cast(float, mb);
    const ToDigits<ND> digits(mx);
    uint32_t w[ND] = {};
    int sum = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int v = digits(x[j]);
        sum += v;
#pragma unroll
        for (int d = 0; d < ND; ++d) w[d] |= digit_of((uint32_t)v + Digits<ND>::kBias, d) << (4 * j);
    }
    sum += __shfl_xor(sum, 1);
    sum += __shfl_xor(sum, 2);
    if (in) {
        uint32_t* o = out + row * digit_row_words<ND>(a.kp);
#pragma unroll
        for (int d = 0; d < ND; ++d) o[d * per + k8] = w[d];
        if ((k8 & 3) == 0) {
            float* f = (float*)(o + ND * per);
            f[k8 / 4] = digit_scale<ND>(mx);
            f[per / 4 + k8 / 4] = (float)sum;
        }
    }
}

// ------------------------------------------------------------------ products

template <int GROUP, int ND, int TT, bool W2, bool GU>
__global__ __launch_bounds__(kMdMaxWaves * kWave, TT == 1 ? 3 : 2) void k_moe_dot(MoeDot a) {
    constexpr int NG = kMdPiece / GROUP;          // groups of a piece and row: 16, 8 or 4
    constexpr int FPG = GROUP / 32;               // fields per group
    constexpr int kSzRow = NG + 1;                // words (step | zero << 16) of a row in LDS, padded
    __shared__ uint32_t sz[kMdMaxWaves][kMdRows * kSzRow];
    __shared__ float red[kMdMaxWaves][TT][kWave];
    const MoeTile tl = a.tiles[blockIdx.y];
    if (tl.count == 0) return;
    const int tid = threadIdx.x, lane = tid & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int nk = a.ksplit, kx = wave % nk, rw = wave / nk, nr = blockDim.x / kWave / nk;
    const int f = lane & 15, g = lane >> 4;
    const int64_t K = a.K, R = GU ? 2 * a.rows : a.rows;
    const int64_t wpr = K / 8, gpr = K / GROUP;
    const int64_t o0 = ((int64_t)blockIdx.x * nr + rw) * (GU ? kMdRows / 2 : kMdRows);
    // Rows past an expert's end (of the last row group) read what follows, or
    // zeros behind the array's end, and are not used.  The first row's offset
    // goes into the descriptors.
    const int64_t base = min(o0, a.rows - 1);
    const int64_t left = R - base;
    const rsrc_t rc = make_rsrc(a.codes + ((int64_t)tl.expert * R + base) * wpr, left * wpr * 4);
    uint32_t sa, za;
    const rsrc_t rsc = moe_half_rsrc(a.scale + ((int64_t)tl.expert * R + base) * gpr, left * gpr * 2, sa);
    const rsrc_t rze = moe_half_rsrc(a.zero + ((int64_t)tl.expert * R + base) * gpr, left * gpr * 2, za);
    const int np = (int)(a.kp / kMdPiece);
    const int pb = (int)blockIdx.z * a.per_slice, pe = min(np, pb + a.per_slice);
    // Byte offsets: code row 4 r + g, field f; steps of row `lane`.
    const uint32_t row4 = (uint32_t)(wpr * 16), up4 = GU ? (uint32_t)((a.rows - 32) * wpr * 4) : 0u;
    const uint32_t co = (uint32_t)(g * wpr * 4 + 16 * f);
    const uint32_t so = (uint32_t)((lane + (GU && lane >= 32 ? a.rows - 32 : 0)) * gpr * 2);

    int slot[TT];
#pragma unroll
    for (int t = 0; t < TT; ++t) slot[t] = a.order[tl.first + min(t, tl.count - 1)];
    u32x4 ring[kMdRing];
    uint32_t sw[NG / 2], zw[NG / 2];
    u32x4 xd[TT][ND];
    float xs[TT], xsum[TT];
    // `at`: co, or an offset behind the buffer (zeros, no traffic) where there
    // is no such piece.  No branch: around the loads it would let the compiler
    // gather all of a piece's products behind them.
    auto load_codes = [&](int r, uint32_t at, int p) __attribute__((always_inline)) {
        ring[r % kMdRing] = __builtin_bit_cast(
            u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                       rc, (int)(at + (r * row4 + (r >= 8 ? up4 : 0u) + (uint32_t)p * (kMdPiece / 2))), 0, 2));
    };
    auto load_steps = [&](int p) __attribute__((always_inline)) {
        const uint32_t off = so + (uint32_t)p * (NG * 2);
        moe_load_halves<NG, W2>(sw, rsc, off + sa);
        moe_load_halves<NG, W2>(zw, rze, off + za);
    };
    auto load_x = [&](int p) __attribute__((always_inline)) {
        const int64_t per = a.kp / 8;
#pragma unroll
        for (int t = 0; t < TT; ++t) {
            const uint32_t* o = a.xq + (slot[t] / a.div) * digit_row_words<ND>(a.kp);
#pragma unroll
            for (int d = 0; d < ND; ++d) xd[t][d] = *(const u32x4*)(o + d * per + (int64_t)p * (kMdPiece / 8) + 4 * f);
            const float* v = (const float*)(o + ND * per) + (int64_t)p * 16 + f;
            xs[t] = v[0];
            xsum[t] = v[per / 4];
        }
    };
    float acc[16][TT];
#pragma unroll
    for (int r = 0; r < 16; ++r)
#pragma unroll
        for (int t = 0; t < TT; ++t) acc[r][t] = 0.f;
    uint32_t* const my = sz[wave];
    int p = pb + kx;
    if (p < pe) {                                 // uniform, as every condition on p below
        load_x(p);
        load_steps(p);
#pragma unroll
        for (int r = 0; r < kMdRing; ++r) load_codes(r, co, p);
    }
    for (; p < pe; p += nk) {
        const int pn = p + nk;
        const uint32_t cn = pn < pe ? co : 0xC0000000u;
        // Steps and zeros of row `lane` to LDS (its reads of the piece before
        // are done: LDS operations of a wave keep their order).
        __builtin_amdgcn_wave_barrier();
        if ((p + 1) * NG > gpr)                   // behind the row: the next row's, which may be anything
#pragma unroll
            for (int v = 0; v < NG / 2; ++v) {
                const uint32_t m = p * NG + 2 * v + 1 < gpr ? 0xFFFFFFFFu : p * NG + 2 * v < gpr ? 0xFFFFu : 0u;
                sw[v] &= m;
                zw[v] &= m;
            }
#pragma unroll
        for (int v = 0; v < NG / 2; ++v) {
            my[lane * kSzRow + 2 * v] = __builtin_amdgcn_perm(zw[v], sw[v], 0x05040100u);
            my[lane * kSzRow + 2 * v + 1] = __builtin_amdgcn_perm(zw[v], sw[v], 0x07060302u);
        }
        __builtin_amdgcn_wave_barrier();
        if (pn < pe) load_steps(pn);
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            u32x4 c = ring[r % kMdRing];
            if (r + kMdRing < 16) load_codes(r + kMdRing, co, p);
            else load_codes(r + kMdRing - 16, cn, pn);
#pragma unroll
            for (int w = 0; w < 4; ++w) c[w] ^= 0x88888888u;
            const uint32_t s = my[(4 * r + g) * kSzRow + f / FPG];
            const float st = half_at(s, false), z8 = 8.f - half_at(s, true);
#pragma unroll
            for (int t = 0; t < TT; ++t) {
                if (t >= tl.count) continue;      // uniform; also keeps the steps apart where TT is 1
                int v = 0;
#pragma unroll
                for (int d = ND - 1; d >= 0; --d) {
                    int dd = 0;
#pragma unroll
                    for (int w = 0; w < 4; ++w) dd = __builtin_amdgcn_sdot8((int)xd[t][d][w], (int)c[w], dd, false);
                    v = (int)((uint32_t)v << 4) + dd;
                }
                acc[r][t] = __builtin_fmaf(st, xs[t] * __builtin_fmaf(z8, xsum[t], (float)v), acc[r][t]);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        if (pn < pe) load_x(pn);
    }

    // Over the 16 fields: lane (g, f) ends with row 4 f + g.
    float tot[TT];
#pragma unroll
    for (int t = 0; t < TT; ++t) {
        float v[16];
#pragma unroll
        for (int r = 0; r < 16; ++r) v[r] = acc[r][t];
#pragma unroll
        for (int m = 8; m >= 1; m >>= 1) {
            const uint32_t um = (f & m) ? 0xFFFFFFFFu : 0u;
#pragma unroll
            for (int i = 0; i < m; ++i) {
                // Selects on the bit patterns: no dynamic array index.
                const uint32_t x = __builtin_bit_cast(uint32_t, v[i]), y = __builtin_bit_cast(uint32_t, v[i + m]);
                const float send = __builtin_bit_cast(float, (x & um) | (y & ~um));
                const float keep = __builtin_bit_cast(float, (y & um) | (x & ~um));
                v[i] = keep + __shfl_xor(send, m);
            }
        }
        tot[t] = v[0];
    }
    if (nk > 1) {                                 // uniform: the waves of a row group in order
#pragma unroll
        for (int t = 0; t < TT; ++t) red[wave][t][lane] = tot[t];
        __syncthreads();
        if (kx != 0) return;
        for (int w = 1; w < nk; ++w)
#pragma unroll
            for (int t = 0; t < TT; ++t) tot[t] += red[wave + w][t][lane];
    }

    if constexpr (!GU) {
        const int64_t o = o0 + 4 * f + g;
#pragma unroll
        for (int t = 0; t < TT; ++t)
            if (t < tl.count && o < a.rows) a.p[((int64_t)blockIdx.z * a.slots + slot[t]) * a.rows + o] = tot[t];
    } else {
        // Lane f < 8: gate row of channel 4 f + g; lane f + 8: its up row.
        // h = act(g) u w / s_down of the wave's 32 channels, as digits.
        const int i = 4 * (f & 7) + g;
        const int64_t o = o0 + i;
        if (o0 >= a.hp) return;                   // uniform
        const int64_t per = a.hp / 8;
#pragma unroll
        for (int t = 0; t < TT; ++t) {
            if (t >= tl.count) continue;
            const float other = __shfl_xor(tot[t], 8);
            const float gate = f < 8 ? tot[t] : other, up = f < 8 ? other : tot[t];
            float h = 0.f;
            if (o < a.rows)
                h = moe_act(gate, a.act) * up * (a.w[slot[t]] / a.s_out[tl.expert * a.s_out_stride + o]);
            uint32_t mb = abs_bits(h);
#pragma unroll
            for (int m = 1; m < kWave; m <<= 1) mb = max(mb, (uint32_t)__shfl_xor((int)mb, m));
            const float mx = __builtin_bit_cast(float, mb);
            const int v = ToDigits<ND>(mx)(h);
            int sum = f < 8 ? v : 0;
#pragma unroll
            for (int m = 1; m < kWave; m <<= 1) sum += __shfl_xor(sum, m);
            uint32_t* q = a.hq + slot[t] * digit_row_words<ND>(a.hp);
#pragma unroll
            for (int d = 0; d < ND; ++d) {
                uint32_t w = digit_of((uint32_t)v + Digits<ND>::kBias, d) << (4 * (i & 7));
                w |= __shfl_xor(w, 1);            // channels 8 c .. 8 c + 7: lane bits 0, 4 and 5
                w |= __shfl_xor(w, 16);
                w |= __shfl_xor(w, 32);
                if (g == 0 && f < 8 && (f & 1) == 0) q[d * per + o0 / 8 + f / 2] = w;
            }
            if (lane == 0) {
                float* s = (float*)(q + ND * per);
                s[o0 / 32] = digit_scale<ND>(mx);
                s[per / 4 + o0 / 32] = (float)sum;
            }
        }
    }
}

// ------------------------------------------------------------------ host

// One slot a tile for one token, two for two; more tokens take the matrix
// cores.
int moe_dot_tile(const ttq_moe_args* a) {
    return a->bits == 4 && a->group >= 32 && a->T <= 2 ? (int)a->T : 0;
}

// Row groups and waves on each one's pieces, up to eight waves a workgroup:
// as many waves as pieces allow until the chip has three per SIMD.
struct MdShape {
    int nr, nk;
};
static MdShape md_shape(int64_t groups, int64_t pieces) {
    MdShape s{1, 1};
    while (s.nk < kMdMaxWaves && s.nk * 2 <= pieces && groups * s.nk < 3 * kSimds) s.nk *= 2;
    while (s.nr * s.nk < 4 && groups / s.nr > 1024) s.nr *= 2;
    return s;
}

// Slices of the second product's pieces over workgroups.
int moe_dot_slices(int64_t n, int64_t E, int64_t I, int64_t M, int tile) {
    const int64_t groups = (M + kMdRows - 1) / kMdRows * moe_tiles(n, E, tile), pieces = moe_dot_pad(I) / kMdPiece;
    if (groups == 0) return 1;                    // an empty call
    int64_t s = (3584 + groups * kMdMaxWaves - 1) / (groups * kMdMaxWaves);
    const int64_t most = (pieces + kMdMaxWaves - 1) / kMdMaxWaves;
    s = s > most ? most : s;
    return (int)(s < 1 ? 1 : s > 16 ? 16 : s);
}

template <int ND, int TT, bool GU>
static hipError_t launch_dot(const MoeDot& p, int group, dim3 grid, int waves, hipStream_t st) {
    const bool w2 = moe_w2(p.scale, p.zero, p.K / group);
#define TTQ_MD(G)                                                                                                   \
    return w2 ? launch_kernel(k_moe_dot<G, ND, TT, true, GU>, grid, dim3(waves * kWave), 0, st, nullptr, nullptr, p) \
              : launch_kernel(k_moe_dot<G, ND, TT, false, GU>, grid, dim3(waves * kWave), 0, st, nullptr, nullptr, p)
    switch (group) {
        case 32: TTQ_MD(32);
        case 64: TTQ_MD(64);
        case 128: TTQ_MD(128);
    }
#undef TTQ_MD
    return hipErrorInvalidValue;
}

template <bool XF32, int TT>
static hipError_t launch_layer(const ttq_moe_args* a, const MoeLayout& L, char* ws, hipStream_t st) {
    constexpr int ND = md_digits(XF32);
    const int64_t n = a->T * a->topk, kp = moe_dot_pad(a->K), ip = moe_dot_pad(a->I);
    const int64_t nt = moe_tiles(n, a->E, TT);
    MoePlan pl{a->ids, (int)n, (int)a->E, TT, (int)nt, (int32_t*)(ws + L.order), (MoeTile*)(ws + L.tiles)};
    MoePrep pr = moe_prep_of(a, kp);
    uint32_t* xq = (uint32_t*)(ws + L.xt);
    const dim3 pg((unsigned)(1 + (pr.rows * (kp / 8) + kPlanThreads - 1) / kPlanThreads));
    if (hipError_t e = launch_kernel(k_moe_dot_prep<XF32>, pg, dim3(kPlanThreads), 0, st, nullptr, nullptr, pl, pr, xq))
        return e;
    MoeDot p{};
    p.tiles = pl.tiles; p.order = pl.order; p.slots = n;
    p.xq = xq; p.K = a->K; p.kp = kp; p.rows = a->I; p.div = pr.s_stride ? 1 : (int)a->topk;
    p.codes = (const uint32_t*)a->gate_up.codes; p.scale = a->gate_up.scale_f16; p.zero = a->gate_up.zero_f16;
    p.per_slice = (int)(kp / kMdPiece);
    p.w = a->w; p.s_out = a->down.s; p.s_out_stride = a->down.s_stride; p.act = a->act;
    p.hq = (uint32_t*)(ws + L.h); p.hp = ip;
    const int64_t gw = ip / (kMdRows / 2);
    const MdShape g = md_shape(gw * nt, p.per_slice);
    p.ksplit = g.nk;
    if (hipError_t e = launch_dot<ND, TT, true>(p, a->group, dim3((unsigned)((gw + g.nr - 1) / g.nr), (unsigned)nt),
                                                g.nr * g.nk, st))
        return e;
    MoeDot d{};
    d.tiles = pl.tiles; d.order = pl.order; d.slots = n;
    d.xq = p.hq; d.K = a->I; d.kp = ip; d.rows = a->M; d.div = 1;
    d.codes = (const uint32_t*)a->down.codes; d.scale = a->down.scale_f16; d.zero = a->down.zero_f16;
    d.p = (float*)(ws + L.p);
    const int pieces = (int)(ip / kMdPiece), sl = moe_dot_slices(n, a->E, a->I, a->M, TT);
    d.per_slice = (pieces + sl - 1) / sl;
    const int nsl = (pieces + d.per_slice - 1) / d.per_slice;
    const int64_t dw = (a->M + kMdRows - 1) / kMdRows;
    const MdShape v = md_shape(dw * nt * nsl, d.per_slice);
    d.ksplit = v.nk;
    if (hipError_t e = launch_dot<ND, TT, false>(d, a->group,
                                                 dim3((unsigned)((dw + v.nr - 1) / v.nr), (unsigned)nt, (unsigned)nsl),
                                                 v.nr * v.nk, st))
        return e;
    return launch_moe_sum(a, d.p, nsl, st);
}

hipError_t launch_moe_dot(const ttq_moe_args* a, const MoeLayout& L, char* ws, hipStream_t st) {
    if (a->T == 1)
        return a->xt == TTQ_F32 ? launch_layer<true, 1>(a, L, ws, st) : launch_layer<false, 1>(a, L, ws, st);
    return a->xt == TTQ_F32 ? launch_layer<true, 2>(a, L, ws, st) : launch_layer<false, 2>(a, L, ws, st);
}

}  // namespace ttq
