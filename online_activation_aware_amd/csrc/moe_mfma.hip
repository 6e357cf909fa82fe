// The mixture-of-experts layer on the matrix cores: 4-bit codes in groups of
// 32, 64 or 128.
//
// As in the few-token projection (qgemv_gs.hip) codes are never expanded to
// weights: per 32-channel subgroup the matrix cores form
//   P[t][o] = sum_j (16 + q_oj) x~_tj,
// slots as the 16 rows and code rows as the 16 columns of a 16x16x32 MFMA,
// and a group adds step P - step (zero + 16) S_t, S_t = sum_j x~_tj, the
// second term as one fp32 16x16x4 MFMA per 128 channels.  16 + q is a bf16
// number whose low byte is 0x80 + 8 q under the high byte 0x41: two bit
// operations and a byte permute per pair of codes; with 16 instead of 128 as
// the offset, the difference of the two terms loses three bits fewer.
// step (zero + 16) is exact in fp32 (11 by 5 bits).
//
// x~ = x / s (and h for the second product) enters as a sum of NS bf16 terms,
// hi = bf16(x~), then bf16 of what is left: 16 bits for two terms (bf16 X,
// whose own 8 bits one more rounding would nearly double in error), 24 for
// three (fp32 X).  The matrix cores have the room: a step is bound by the
// codes' way from HBM and the integer work of expanding them.  The terms and
// the 32-channel sums are laid out once per row (k_moe_prep; the first
// product's epilogue for h), each 8 channels in the order 0 2 4 6 1 3 5 7
// that the expansion produces, so that a lane loads an operand with one
// 16-byte load.
//
// A workgroup owns 64 code rows (four column tiles; the first product: 32
// gate rows and their 32 up rows) and up to 16 slots of one expert; its waves
// take pairs of 128-channel chunks (256 channels: whole 128-byte lines of
// codes per row) in turn, the next chunk's loads in flight while one is
// multiplied, and their tiles are added in wave order through LDS.  The
// second product's channels can be split further over workgroups (slices);
// the sum over a token's slots adds the slices, too.
#include "common.hpp"
#include "launch.hpp"
#include "lds_dma.hpp"
#include "moe.hpp"

namespace ttq {

constexpr int kMmMaxWaves = 8;
constexpr int kMmRows = 64;                       // code rows per workgroup
constexpr int kMmChunk = 128;

int64_t moe_pad(int64_t K) { return (K + kMmChunk - 1) / kMmChunk * kMmChunk; }

bool moe_mfma_ok(const ttq_moe_args* a) {
    const int64_t lim = (int64_t)1 << 31;
    return a->bits == 4 && a->group >= 32 && 2 * a->I * a->K / 2 < lim && a->M * a->I / 2 < lim;
}

// ------------------------------------------------------------------ operand layout

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
template <int NS, bool XF32>
__global__ __launch_bounds__(kPlanThreads) void k_moe_prep(MoePlan pl, MoePrep a) {
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
    if (use) {
        if constexpr (XF32) {
            const f32x4 u = *(const f32x4*)((const float*)a.X + t * a.ldx + k0);
            const f32x4 v = *(const f32x4*)((const float*)a.X + t * a.ldx + k0 + 4);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                x[j] = u[j];
                x[4 + j] = v[j];
            }
        } else {
            const u32x4 u = *(const u32x4*)((const uint16_t*)a.X + t * a.ldx + k0);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                x[2 * j] = bf16lo_to_f32(u[j]);
                x[2 * j + 1] = bf16hi_to_f32(u[j]);
            }
        }
        const float* s = a.s + e * a.s_stride + k0;
        const f32x4 u = *(const f32x4*)s, v = *(const f32x4*)(s + 4);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            x[j] /= u[j];
            x[4 + j] /= v[j];
        }
    }
    float sum = 0.f;
    if (in) sum = store_terms<NS>(x, a.xt + row * NS * a.kp + k0, a.kp);
    sum += __shfl_xor(sum, 1);
    sum += __shfl_xor(sum, 2);
    if (in && (threadIdx.x & 3) == 0) a.xs[row * (a.kp / 32) + k0 / 32] = sum;
}

// ------------------------------------------------------------------ products

// The bf16 numbers 16 + q of the eight codes of a word, slot order 0 2 4 6 1 3 5 7.
__device__ __forceinline__ u32x4 codes_plus16(uint32_t w) {
    const uint32_t lo = ((w << 3) & 0x78787878u) | 0x80808080u, hi = ((w >> 1) & 0x78787878u) | 0x80808080u;
    constexpr uint32_t k41 = 0x41414141u;
    return u32x4{__builtin_amdgcn_perm(k41, lo, 0x04010400u), __builtin_amdgcn_perm(k41, lo, 0x04030402u),
                 __builtin_amdgcn_perm(k41, hi, 0x04010400u), __builtin_amdgcn_perm(k41, hi, 0x04030402u)};
}

// 4x4 exchange between the lane quarters and the four words of a lane: word
// j of quarter q becomes word q of quarter j.
__device__ __forceinline__ void exchange_quarters(u32x4& w) {
    const auto a = __builtin_amdgcn_permlane32_swap(w[0], w[2], false, false);
    const auto b = __builtin_amdgcn_permlane32_swap(w[1], w[3], false, false);
    const auto c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
    const auto d = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
    w = u32x4{c[0], c[1], d[0], d[1]};
}

template <int GROUP, int NS>
struct MmStage {
    static constexpr int NG = kMmChunk / GROUP;   // groups per chunk
    u32x4 cw[4];
    uint32_t sw[4][(NG + 1) / 2], zw[4][(NG + 1) / 2];
    u32x4 xa[NS][4];
    float si;
};

// NG fp16 values at byte offset `off` as packed words; W2: two-byte loads
// (rows of the array that are aligned to nothing more).
template <int NG, bool W2>
__device__ __forceinline__ void load_groups(uint32_t (&d)[(NG + 1) / 2], rsrc_t r, uint32_t off) {
    if constexpr (NG == 1) {
        d[0] = __builtin_amdgcn_raw_buffer_load_b16(r, (int)off, 0, 0);
    } else if constexpr (W2) {
#pragma unroll
        for (int v = 0; v < NG / 2; ++v)
            d[v] = (uint32_t)__builtin_amdgcn_raw_buffer_load_b16(r, (int)(off + 4 * v), 0, 0) |
                   ((uint32_t)__builtin_amdgcn_raw_buffer_load_b16(r, (int)(off + 4 * v + 2), 0, 0) << 16);
    } else if constexpr (NG == 2) {
        d[0] = __builtin_amdgcn_raw_buffer_load_b32(r, (int)off, 0, 0);
    } else {
        const u32x2 a = __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(r, (int)off, 0, 0));
        d[0] = a[0];
        d[1] = a[1];
    }
}

__device__ __forceinline__ float half_of(uint32_t d, bool hi) { return f16_to_f32((uint16_t)(hi ? d >> 16 : d & 0xFFFFu)); }

template <int GROUP, int NS, bool W2, bool GU>
__global__ __launch_bounds__(kMmMaxWaves * kWave) void k_moe_mfma(MoeMm a) {
    constexpr int NG = kMmChunk / GROUP;
    constexpr int SPG = GROUP / 32;               // subgroups per group
    __shared__ f32x4 red[kMmMaxWaves][4][kWave];
    const MoeTile tl = a.tiles[blockIdx.y];
    if (tl.count == 0) return;
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int nw = blockDim.x / kWave;
    const int r16 = lane & 15, q = lane >> 4;
    const int64_t K = a.K, R = GU ? 2 * a.rows : a.rows;
    const int64_t wpr = K / 8, gpr = K / GROUP;
    const int64_t o0 = (int64_t)blockIdx.x * (GU ? kMmRows / 2 : kMmRows);
    const rsrc_t rc = make_rsrc(a.codes + (int64_t)tl.expert * R * wpr, R * wpr * 4);
    const rsrc_t rsc = make_rsrc(a.scale + (int64_t)tl.expert * R * gpr, R * gpr * 2);
    const rsrc_t rze = make_rsrc(a.zero + (int64_t)tl.expert * R * gpr, R * gpr * 2);
    // Row of this lane in each column tile; rows past the end are clamped and
    // their outputs not used.
    uint32_t co[4], go[4];
#pragma unroll
    for (int rt = 0; rt < 4; ++rt) {
        int64_t o;
        if constexpr (GU) o = min(o0 + 16 * (rt & 1) + r16, a.rows - 1) + (rt >= 2 ? a.rows : 0);
        else o = min(o0 + 16 * rt + r16, a.rows - 1);
        co[rt] = (uint32_t)(o * wpr * 4 + 16 * q);
        go[rt] = (uint32_t)(o * gpr * 2);
    }
    // Slot of this lane's row of the token operand (lanes past the tile's
    // slots repeat its first one; their outputs are not used).
    const int slot = a.order[tl.first + (r16 < tl.count ? r16 : 0)];
    const int64_t xrow = slot / a.div;
    // In quarter q, MFMA j takes channels 32 j + 8 q ..+7 of the chunk (the
    // codes after the exchange of quarters), with one group per chunk
    // 32 q + 8 j ..+7 (no exchange needed).
    constexpr int kXq = GROUP < 128 ? 8 : 32, kXj = GROUP < 128 ? 32 : 8;
    const uint16_t* xp = a.xt + xrow * NS * a.kp + kXq * q;
    const float* sp = a.xs + xrow * (a.kp / 32) + q;

    // Chunks of this slice, in pairs; pair p of the slice belongs to wave
    // p % nw.  cnt: this wave's chunks.
    const int nch = (int)(a.kp / kMmChunk);
    const int cb = (int)blockIdx.z * a.per_slice;
    const int ce = min(nch, cb + a.per_slice);
    auto chunk = [&](int i) { return cb + 2 * ((i >> 1) * nw + wave) + (i & 1); };
    int cnt = 0;
    if (const int left = ce - cb - 2 * wave; left > 0) {
        const int full = left / (2 * nw), rest = left - full * 2 * nw;
        cnt = 2 * full + min(rest, 2);
    }

    f32x4 acc[4];
#pragma unroll
    for (int rt = 0; rt < 4; ++rt) acc[rt] = f32x4{0.f, 0.f, 0.f, 0.f};

    auto load = [&](MmStage<GROUP, NS>& s, int i) __attribute__((always_inline)) {
        const uint32_t c = (uint32_t)chunk(i);
#pragma unroll
        for (int rt = 0; rt < 4; ++rt)
            s.cw[rt] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rc, (int)(co[rt] + c * 64), 0, 2));
#pragma unroll
        for (int rt = 0; rt < 4; ++rt) {
            load_groups<NG, W2>(s.sw[rt], rsc, go[rt] + c * (NG * 2));
            load_groups<NG, W2>(s.zw[rt], rze, go[rt] + c * (NG * 2));
        }
#pragma unroll
        for (int n = 0; n < NS; ++n)
#pragma unroll
            for (int j = 0; j < 4; ++j) s.xa[n][j] = *(const u32x4*)(xp + n * a.kp + c * kMmChunk + kXj * j);
        s.si = sp[c * 4];
    };
    auto multiply = [&](const MmStage<GROUP, NS>& s) __attribute__((always_inline)) {
#pragma unroll
        for (int rt = 0; rt < 4; ++rt) {
            u32x4 w = s.cw[rt];
            if constexpr (GROUP < 128) exchange_quarters(w);
            f32x4 p = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const u32x4 b = codes_plus16(w[j]);
#pragma unroll
                for (int n = NS - 1; n >= 0; --n) p = mfma_16x16x32(s.xa[n][j], b, p);
                if ((j + 1) % SPG == 0) {
                    const int g = j / SPG;
                    const float st = half_of(s.sw[rt][g / 2], g & 1);
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[rt][e] = __builtin_fmaf(st, p[e], acc[rt][e]);
                    p = f32x4{0.f, 0.f, 0.f, 0.f};
                }
            }
            // step (zero + 16) of the group of subgroup q.
            uint32_t sd = s.sw[rt][0], zd = s.zw[rt][0];
            bool hi = false;
            if constexpr (NG == 4) {
                sd = q >= 2 ? s.sw[rt][1] : sd;
                zd = q >= 2 ? s.zw[rt][1] : zd;
                hi = q & 1;
            } else if constexpr (NG == 2) {
                hi = q >= 2;
            }
            const float nb = -(half_of(sd, hi) * (half_of(zd, hi) + 16.f));
            acc[rt] = __builtin_amdgcn_mfma_f32_16x16x4f32(s.si, nb, acc[rt], 0, 0, 0);
        }
    };
    if (cnt > 0) {                                // as every condition on cnt below: wave-uniform
        MmStage<GROUP, NS> s0, s1;
        load(s0, 0);
        for (int i = 0; i < cnt; i += 2) {
            if (i + 1 < cnt) load(s1, i + 1);
            __builtin_amdgcn_sched_barrier(0);
            multiply(s0);
            if (i + 1 >= cnt) break;
            if (i + 2 < cnt) load(s0, i + 2);
            __builtin_amdgcn_sched_barrier(0);
            multiply(s1);
        }
    }

    // Lane: slots 4 q + e of row r16 of each column tile.  Waves added in
    // wave order.
#pragma unroll
    for (int rt = 0; rt < 4; ++rt) red[wave][rt][lane] = acc[rt];
    __syncthreads();
    const int nsum = GU ? 2 : 4;
    f32x4 sum[2];
    for (int rt = wave; rt < nsum; rt += nw) {
#pragma unroll
        for (int b = 0; b < (GU ? 2 : 1); ++b) {
            f32x4 v = red[0][rt + 2 * b][lane];
            for (int w = 1; w < nw; ++w) {
                const f32x4 u = red[w][rt + 2 * b][lane];
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] += u[e];
            }
            sum[b] = v;
        }
        if constexpr (!GU) {
            const int64_t o = o0 + 16 * rt + r16;
            if (o < a.rows) {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (4 * q + e < tl.count)
                        a.p[((int64_t)blockIdx.z * a.slots + a.order[tl.first + 4 * q + e]) * a.rows + o] = sum[0][e];
            }
        } else {
            // h = act(g) u w / s_down of 4 slots and one channel, into the
            // gate tile's part of red (read by this wave alone so far).
            const int64_t o = o0 + 16 * rt + r16;
            f32x4 h;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int t = 4 * q + e;
                h[e] = 0.f;
                if (o < a.rows && t < tl.count) {
                    const float f = a.w[a.order[tl.first + t]] / a.s_out[tl.expert * a.s_out_stride + o];
                    h[e] = moe_act(sum[0][e], a.act) * sum[1][e] * f;
                }
            }
            red[0][rt][lane] = h;
        }
    }
    if constexpr (GU) {
        // The 32 channels of 16 slots as the second product's operand: thread
        // (slot, 8 channels).
        __syncthreads();
        if (wave == 0) {
            const int t = lane >> 2, c8 = lane & 3;   // channels 8 c8 ..+7: rows 8 (c8 & 1) ..+7 of tile c8 / 2
            float x[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float* v = (const float*)&red[0][c8 >> 1][16 * (t >> 2) + 8 * (c8 & 1) + e];
                x[e] = v[t & 3];
            }
            const bool in = t < tl.count;
            const int64_t hs = a.order[tl.first + (in ? t : 0)];
            float s = 0.f;
            if (in) s = store_terms<NS>(x, a.ht + hs * NS * a.hp + o0 + 8 * c8, a.hp);
            s += __shfl_xor(s, 1);
            s += __shfl_xor(s, 2);
            if (in && c8 == 0) a.hs[hs * (a.hp / 32) + o0 / 32] = s;
        }
    }
}

// ------------------------------------------------------------------ host

// Waves of a workgroup: one per pair of chunks, at most eight.
static int mm_waves(int64_t chunks) {
    const int64_t p = (chunks + 1) / 2;
    return (int)(p < kMmMaxWaves ? p : kMmMaxWaves);
}

// Slices of the second product's channels: enough workgroups for every
// compute unit, at least 16 chunks (a round of eight waves) each.
int moe_slices(int64_t n, int64_t E, int64_t I, int64_t M) {
    const int64_t tiles = moe_tiles(n, E, kMmTile), wgs = (M + kMmRows - 1) / kMmRows * tiles;
    const int64_t chunks = moe_pad(I) / kMmChunk, most = chunks / 16 > 0 ? chunks / 16 : 1;
    if (wgs == 0) return 1;                       // an empty call
    int64_t s = (512 + wgs - 1) / wgs;
    if (s > most) s = most;
    return (int)(s < 1 ? 1 : s > 16 ? 16 : s);
}

template <int NS, bool GU>
static hipError_t launch_mm(const MoeMm& p, int group, dim3 grid, int waves, hipStream_t st) {
    const bool w2 = p.K % 128 != 0;
#define TTQ_MM(G)                                                                                                     \
    return w2 ? launch_kernel(k_moe_mfma<G, NS, true, GU>, grid, dim3(waves * kWave), 0, st, nullptr, nullptr, p)     \
              : launch_kernel(k_moe_mfma<G, NS, false, GU>, grid, dim3(waves * kWave), 0, st, nullptr, nullptr, p)
    switch (group) {
        case 32: TTQ_MM(32);
        case 64: TTQ_MM(64);
        case 128: TTQ_MM(128);
    }
#undef TTQ_MM
    return hipErrorInvalidValue;
}

template <int NS>
static hipError_t launch_ns(const ttq_moe_args* a, const MoeLayout& L, char* ws, hipStream_t st) {
    const int64_t n = a->T * a->topk, kp = moe_pad(a->K), ip = moe_pad(a->I);
    const int64_t nt = moe_tiles(n, a->E, kMmTile);
    MoePlan pl{a->ids, (int)n, (int)a->E, kMmTile, (int)nt, (int32_t*)(ws + L.order), (MoeTile*)(ws + L.tiles)};
    MoePrep pr{};
    pr.X = a->X; pr.ldx = a->ldx; pr.K = a->K; pr.kp = kp;
    pr.s = a->gate_up.s; pr.s_stride = a->gate_up.s_stride;
    pr.rows = pr.s_stride ? n : a->T; pr.ids = a->ids; pr.topk = (int)a->topk; pr.E = (int)a->E;
    pr.xt = (uint16_t*)(ws + L.xt); pr.xs = (float*)(ws + L.xs);
    const dim3 pg((unsigned)(1 + (pr.rows * (kp / 8) + kPlanThreads - 1) / kPlanThreads));
    if (hipError_t e = a->xt == TTQ_F32
                           ? launch_kernel(k_moe_prep<NS, true>, pg, dim3(kPlanThreads), 0, st, nullptr, nullptr, pl, pr)
                           : launch_kernel(k_moe_prep<NS, false>, pg, dim3(kPlanThreads), 0, st, nullptr, nullptr, pl, pr))
        return e;
    MoeMm p{};
    p.tiles = pl.tiles; p.order = pl.order; p.slots = n;
    p.xt = pr.xt; p.xs = pr.xs; p.K = a->K; p.kp = kp; p.rows = a->I; p.div = pr.s_stride ? 1 : (int)a->topk;
    p.codes = (const uint32_t*)a->gate_up.codes; p.scale = a->gate_up.scale_f16; p.zero = a->gate_up.zero_f16;
    p.per_slice = (int)(kp / kMmChunk);
    p.w = a->w; p.s_out = a->down.s; p.s_out_stride = a->down.s_stride; p.act = a->act;
    p.ht = (uint16_t*)(ws + L.h); p.hs = (float*)(ws + L.hs); p.hp = ip;
    if (hipError_t e = launch_mm<NS, true>(p, a->group, dim3((unsigned)(ip / 32), (unsigned)nt), mm_waves(p.per_slice), st))
        return e;
    MoeMm d{};
    d.tiles = pl.tiles; d.order = pl.order; d.slots = n;
    d.xt = p.ht; d.xs = p.hs; d.K = a->I; d.kp = ip; d.rows = a->M; d.div = 1;
    d.codes = (const uint32_t*)a->down.codes; d.scale = a->down.scale_f16; d.zero = a->down.zero_f16;
    d.p = (float*)(ws + L.p);
    const int sl = moe_slices(n, a->E, a->I, a->M);
    const int chunks = (int)(ip / kMmChunk);
    d.per_slice = ((chunks + sl - 1) / sl + 1) / 2 * 2;
    const int nsl = (chunks + d.per_slice - 1) / d.per_slice;
    if (hipError_t e = launch_mm<NS, false>(d, a->group,
                                            dim3((unsigned)((a->M + kMmRows - 1) / kMmRows), (unsigned)nt, (unsigned)nsl),
                                            mm_waves(d.per_slice), st))
        return e;
    return launch_moe_sum(a, d.p, nsl, st);
}

hipError_t launch_moe_mfma(const ttq_moe_args* a, const MoeLayout& L, char* ws, hipStream_t st) {
    return a->xt == TTQ_F32 ? launch_ns<3>(a, L, ws, st) : launch_ns<2>(a, L, ws, st);
}

}  // namespace ttq
