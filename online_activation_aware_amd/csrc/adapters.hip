// Low-rank adapters of many requests at once:
//   Y[t] = C[t] + scale_a B_a (A_a x_t),   a = ids[t],
// where A_a is the adapter's first r_a rows of [rank][K], B_a the first r_a
// columns of [M][rank]; a token whose id names no adapter gets C[t] itself.
//
// Two launches of matrix-core kernels: z[t][k] = sum_j A[a][k][j] x[t][j]
// (fp32, K slices as partial sums into the workspace), then Y.  Tokens come
// in tiles of 16, the columns of 16x16 MFMAs; a wave finds the distinct
// adapters of its tile by ballots over the tokens' ids and makes one product
// per adapter, of which the adapter's own tokens keep their columns: 16
// requests of 16 adapters read each adapter once, a prompt's tile one.  What
// lies behind an adapter's rank is loaded as zero (through the bounds of the
// buffer), so that it may hold anything.
//
// bf16 operands are multiplied as they are (products exact, fp32 sums); z is
// split into three bf16 terms against a bf16 B (24 bits).  With an fp32
// operand both products are fp32 MFMAs.
#include "common.hpp"
#include "launch.hpp"
#include "lds_dma.hpp"

namespace ttq {

constexpr uint32_t kOut = 0x80000000u;            // an offset behind every buffer: loads return zero

// Rows of adapter a in use; 0 where the id names none.
__device__ __forceinline__ int adapter_rank(const AdapterTable& ad, int a) {
    if (a < 0 || a >= ad.n) return 0;
    if (ad.ranks == nullptr) return ad.rank;
    const int r = ad.ranks[a];
    return r < 0 ? 0 : r > ad.rank ? ad.rank : r;
}

// 8 consecutive values at an element offset of a buffer: 4 words of bf16
// pairs, or 8 of fp32.
template <bool F32>
struct Eight {
    uint32_t w[F32 ? 8 : 4];
};
template <bool F32>
__device__ __forceinline__ Eight<F32> load_eight(rsrc_t r, uint32_t off) {   // bytes, 16-byte aligned (or 4)
    Eight<F32> v;
#pragma unroll
    for (int h = 0; h < (F32 ? 2 : 1); ++h) {
        const u32x4 a = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, (int)(off + 16 * h), 0, 0));
#pragma unroll
        for (int e = 0; e < 4; ++e) v.w[4 * h + e] = a[e];
    }
    return v;
}
template <bool F32>
__device__ __forceinline__ float eight_at(const Eight<F32>& v, int e) {
    if constexpr (F32) return __builtin_bit_cast(float, v.w[e]);
    else return (e & 1) ? bf16hi_to_f32(v.w[e / 2]) : bf16lo_to_f32(v.w[e / 2]);
}

// acc += U V^T over 32 slots: lane (r16, q) holds 8 slots of row r16 of each.
template <bool F32A, bool F32B>
__device__ __forceinline__ f32x4 mac32(const Eight<F32A>& u, const Eight<F32B>& v, f32x4 acc) {
    if constexpr (!F32A && !F32B) {
        return mfma_16x16x32(u32x4{u.w[0], u.w[1], u.w[2], u.w[3]}, u32x4{v.w[0], v.w[1], v.w[2], v.w[3]}, acc);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            acc = __builtin_amdgcn_mfma_f32_16x16x4f32(eight_at<F32A>(u, e), eight_at<F32B>(v, e), acc, 0, 0, 0);
        return acc;
    }
}

// The distinct adapters of a tile of 16 tokens (lane r16: token id and rank)
// into LDS by the first wave: list and ranks in `dist` and `dr`, each token's
// place in the list, or -1, in `dof`.  Returns their number, in every wave.
__device__ __forceinline__ int tile_adapters(int id, int rk, int* dist, int* dr, int* dof) {
    int nd = 0, place = -1;
    uint32_t left = (uint32_t)__ballot(rk > 0) & 0xFFFFu;
    while (left) {                                // at most 16 rounds: each takes its first token's bit
        const int f = __builtin_ctz(left);
        const int a = __builtin_amdgcn_readlane(id, f), r = __builtin_amdgcn_readlane(rk, f);
        const bool mine = rk > 0 && id == a;
        left &= ~((uint32_t)__ballot(mine) & 0xFFFFu);
        if (mine) place = nd;
        if (threadIdx.x == 0) {
            dist[nd] = a;
            dr[nd] = r;
        }
        ++nd;
    }
    if (threadIdx.x < 16) dof[threadIdx.x] = place;
    return nd;
}

// ------------------------------------------------------------------ z

// A workgroup owns 16 tokens and one K slice; its items (distinct adapter d,
// part c of the slice) go to the waves, C parts per adapter so that few
// adapters still use all of them.  RT: 16-row tiles of the rank.
constexpr int kAzWaves = 8;

template <bool XF32, bool AF32, int RT>
__global__ __launch_bounds__(kAzWaves * kWave) void k_adapter_z(const void* __restrict__ X, int64_t T, int64_t K,
                                                                int64_t ldx, AdapterTable ad, int64_t per,
                                                                float* __restrict__ Z) {
    __shared__ f32x4 red[kAzWaves][RT][kWave];
    __shared__ int dist[16], dr[16], dof[16];
    constexpr int XE = XF32 ? 4 : 2, AE = AF32 ? 4 : 2;
    const int tid = threadIdx.x, lane = tid & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int r16 = lane & 15, q = lane >> 4;
    const int64_t t0 = (int64_t)blockIdx.x * 16;
    const int rows = (int)min((int64_t)16, T - t0);
    const int64_t k0 = (int64_t)blockIdx.y * per, k1 = min(K, k0 + per);
    const int id = r16 < rows ? ad.ids[t0 + r16] : -1;
    const int rk = adapter_rank(ad, id);
    const int nd = tile_adapters(id, rk, dist, dr, dof);
    __syncthreads();
    const int parts = nd == 0 ? 1 : kAzWaves / nd > 0 ? kAzWaves / nd : 1;
    const int64_t steps = (k1 - k0 + 31) / 32, sp = (steps + parts - 1) / parts;
    const rsrc_t rx = make_rsrc((const char*)X + t0 * ldx * XE, ((rows - 1) * ldx + K) * XE);
    const int R = ad.rank;
    // Items in rounds of one per wave; after a round its adapters' sums go out.
    for (int base = 0; base < nd * parts; base += kAzWaves) {
        const int item = base + wave, d = item / parts, c = item - d * parts;
        f32x4 acc[RT];
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) acc[rt] = f32x4{0.f, 0.f, 0.f, 0.f};
        if (item < nd * parts) {
            const int a = __builtin_amdgcn_readfirstlane(dist[d]);
            const int ra = __builtin_amdgcn_readfirstlane(dr[d]);
            const rsrc_t rA = make_rsrc((const char*)ad.A + (int64_t)a * R * K * AE, (int64_t)ra * K * AE);
            const int64_t sb = c * sp, se = min(steps, sb + sp);
            constexpr int U = RT >= 4 ? 2 : 4;    // steps whose loads are in flight together
            for (int64_t s0 = sb; s0 < se; s0 += U) {
                Eight<XF32> x[U];
                Eight<AF32> w[U][RT];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int64_t j = k0 + (s0 + u) * 32 + 8 * q;   // K % 8 == 0: all in or all out
                    const bool in = s0 + u < se && j < k1;
                    x[u] = load_eight<XF32>(rx, in && r16 < rows ? (uint32_t)((r16 * ldx + j) * XE) : kOut);
#pragma unroll
                    for (int rt = 0; rt < RT; ++rt)
                        w[u][rt] = load_eight<AF32>(rA, in ? (uint32_t)(((16 * rt + r16) * K + j) * AE) : kOut);
                }
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                    for (int rt = 0; rt < RT; ++rt) acc[rt] = mac32<AF32, XF32>(w[u][rt], x[u], acc[rt]);
            }
        }
        if (base > 0) __syncthreads();
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) red[wave][rt][lane] = acc[rt];
        __syncthreads();
        // Lane of tile rt: z^T[16 rt + 4 q + i][r16], parts in order.
        for (int rt = wave; rt < RT; rt += kAzWaves) {
            const int d0 = base / parts, pl = dof[r16];
            if (pl >= d0 && pl < d0 + kAzWaves / parts) {
                f32x4 z = red[(pl - d0) * parts][rt][lane];
                for (int w = 1; w < parts; ++w) {
                    const f32x4 v = red[(pl - d0) * parts + w][rt][lane];
#pragma unroll
                    for (int i = 0; i < 4; ++i) z[i] += v[i];
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int k = 16 * rt + 4 * q + i;
                    if (k < R) Z[((int64_t)blockIdx.y * T + t0 + r16) * R + k] = z[i];
                }
            }
        }
    }
}

// ------------------------------------------------------------------ Y

// A wave owns 16 tokens and RT 16-row tiles of M at a time; workgroup: 4
// waves on the same tokens.  VEC: rows of B and of C and Y allow 16-byte
// (B) and 4-value (C, Y) accesses.  ST: 32-slot steps of the rank.
constexpr int kAyWaves = 4;

// Four consecutive values of C (zeros without C) as fp32.
template <bool CF32>
__device__ __forceinline__ f32x4 load_c4(const void* C, int64_t i, int64_t avail, bool vec) {
    f32x4 v = f32x4{0.f, 0.f, 0.f, 0.f};
    if (C == nullptr || avail <= 0) return v;
    if (vec && avail >= 4) {
        if constexpr (CF32) return *(const f32x4*)((const float*)C + i);
        const u32x2 c = *(const u32x2*)((const uint16_t*)C + i);
        return f32x4{bf16lo_to_f32(c[0]), bf16hi_to_f32(c[0]), bf16lo_to_f32(c[1]), bf16hi_to_f32(c[1])};
    }
#pragma unroll
    for (int r = 0; r < 4; ++r)
        if (r < avail) {
            if constexpr (CF32) v[r] = ((const float*)C)[i + r];
            else v[r] = bf16_to_f32(((const uint16_t*)C)[i + r]);
        }
    return v;
}

template <bool BF32, bool VEC>
__device__ __forceinline__ Eight<BF32> load_b(rsrc_t r, int row, int k, int ra, int R, bool in) {
    constexpr int BE = BF32 ? 4 : 2;
    const uint32_t off = (uint32_t)((row * R + k) * BE);
    Eight<BF32> v;
    if constexpr (VEC) {                          // R % 8 == 0: 8 columns are all in the row
        v = load_eight<BF32>(r, in && k < ra ? off : kOut);
        if (ra & 7) {                             // uniform: columns behind the rank as zeros
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (k + e >= ra) {
                    if constexpr (BF32) v.w[e] = 0u;
                    else v.w[e / 2] &= (e & 1) ? 0x0000FFFFu : 0xFFFF0000u;
                }
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const uint32_t o = in && k + e < ra ? off + BE * e : kOut;
            if constexpr (BF32) {
                v.w[e] = __builtin_amdgcn_raw_buffer_load_b32(r, (int)o, 0, 0);
            } else {
                const uint32_t h = (uint32_t)__builtin_amdgcn_raw_buffer_load_b16(r, (int)o, 0, 0);
                v.w[e / 2] = (e & 1) ? v.w[e / 2] | (h << 16) : h;
            }
        }
    }
    return v;
}

// acc += B z over a step: z as three bf16 terms (bf16 B), or fp32.
template <bool BF32>
struct ZOp {
    u32x4 t[BF32 ? 2 : 3];
};
template <bool BF32>
__device__ __forceinline__ ZOp<BF32> z_operand(const float (&z)[8]) {
    ZOp<BF32> o;
    if constexpr (BF32) {
#pragma unroll
        for (int e = 0; e < 8; ++e) o.t[e / 4][e % 4] = __builtin_bit_cast(uint32_t, z[e]);
    } else {
        float x[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = z[e];
#pragma unroll
        for (int n = 0; n < 3; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t p = pack_bf16x2(x[2 * e], x[2 * e + 1]);
                o.t[n][e] = p;
                x[2 * e] -= bf16lo_to_f32(p);
                x[2 * e + 1] -= bf16hi_to_f32(p);
            }
    }
    return o;
}
template <bool BF32>
__device__ __forceinline__ f32x4 mac_z(const Eight<BF32>& b, const ZOp<BF32>& z, f32x4 acc) {
    if constexpr (BF32) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const uint32_t v = z.t[e / 4][e % 4];   // a bit cast of the vector's element itself reads element 0
            acc = __builtin_amdgcn_mfma_f32_16x16x4f32(eight_at<true>(b, e), __builtin_bit_cast(float, v), acc, 0, 0, 0);
        }
    } else {
        const u32x4 v = {b.w[0], b.w[1], b.w[2], b.w[3]};
#pragma unroll
        for (int n = 2; n >= 0; --n) acc = mfma_16x16x32(v, z.t[n], acc);
    }
    return acc;
}

template <bool CF32, bool BF32, bool YF32, bool VEC, int RT, int ST>
__global__ __launch_bounds__(kAyWaves * kWave) void k_adapter_y(const float* __restrict__ Z, int slices, int64_t T,
                                                                AdapterTable ad, const void* C, int64_t ldc, int64_t M,
                                                                void* Y, int64_t ldy, int blocks, int cvec, int yvec) {
    constexpr int BE = BF32 ? 4 : 2;
    constexpr int U = RT == 1 ? 4 : 1;            // adapters whose rows are in flight together
    constexpr int kZRow = 32 * ST + 4;
    __shared__ __attribute__((aligned(16))) float zl[16][kZRow];
    __shared__ int dist[16], dr[16], dof[16];
    const int tid = threadIdx.x, lane = tid & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int r16 = lane & 15, q = lane >> 4;
    const int64_t t0 = (int64_t)blockIdx.x * 16, t = t0 + r16;
    const int R = ad.rank;
    const int id = t < T ? ad.ids[t] : -1;
    const int rk = adapter_rank(ad, id);
    const int nd = tile_adapters(id, rk, dist, dr, dof);
    // z of the tile, slices in order, times the adapters' scales.
    {
        const int zt = tid & 15;                  // 16 threads on each token's ranks
        const int zr = __shfl(rk, zt);            // every wave's lanes 0..15 hold the tokens
        const float sc = zr > 0 && ad.scale != nullptr ? ad.scale[__shfl(id, zt)] : 1.f;
        const int64_t step = T * R;
        for (int k = tid >> 4; k < 32 * ST; k += kAyWaves * kWave / 16) {
            float v = 0.f;
            if (k < zr) {
                const float* p = Z + (t0 + zt) * R + k;
                int i = 0;
                for (; i + 8 <= slices; i += 8) {
                    float x[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) x[j] = p[(i + j) * step];
#pragma unroll
                    for (int j = 0; j < 8; ++j) v += x[j];
                }
                for (; i < slices; ++i) v += p[i * step];
            }
            zl[zt][k] = v * sc;
        }
    }
    __syncthreads();
    ZOp<BF32> zo[ST];
#pragma unroll
    for (int s = 0; s < ST; ++s) {
        float z[8];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const f32x4 v = *(const f32x4*)&zl[r16][32 * s + 8 * q + 4 * h];
#pragma unroll
            for (int e = 0; e < 4; ++e) z[4 * h + e] = v[e];
        }
        zo[s] = z_operand<BF32>(z);
    }
    const int place = dof[r16];
    // `blocks` row blocks of 16 RT kAyWaves rows per workgroup.
    for (int bi = 0; bi < blocks; ++bi) {
        const int64_t o0 = (((int64_t)blockIdx.y * blocks + bi) * kAyWaves + wave) * (16 * RT);
        if (o0 >= M) break;
        f32x4 acc[RT], c[RT];
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
            const int64_t o = o0 + 16 * rt + 4 * q;
            acc[rt] = f32x4{0.f, 0.f, 0.f, 0.f};
            c[rt] = load_c4<CF32>(C, t * ldc + o, t < T ? M - o : 0, cvec);
        }
        for (int d0 = 0; d0 < nd; d0 += U) {
            Eight<BF32> b[U][RT][ST];
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (d0 + u < nd) {                // uniform
                    const int a = __builtin_amdgcn_readfirstlane(dist[d0 + u]);
                    const int ra = __builtin_amdgcn_readfirstlane(dr[d0 + u]);
                    const rsrc_t rB = make_rsrc((const char*)ad.B + ((int64_t)a * M + o0) * R * BE,
                                                min((int64_t)16 * RT, M - o0) * R * BE);
#pragma unroll
                    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
                        for (int s = 0; s < ST; ++s) {
                            const int r = 16 * rt + r16;
                            b[u][rt][s] = load_b<BF32, VEC>(rB, r, 32 * s + 8 * q, ra, R, o0 + r < M);
                        }
                }
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (d0 + u < nd) {
                    const bool mine = place == d0 + u;
#pragma unroll
                    for (int rt = 0; rt < RT; ++rt) {
                        f32x4 p = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                        for (int s = 0; s < ST; ++s) p = mac_z<BF32>(b[u][rt][s], zo[s], p);
#pragma unroll
                        for (int e = 0; e < 4; ++e) acc[rt][e] = mine ? p[e] : acc[rt][e];
                    }
                }
        }
        // Lane: rows 16 rt + 4 q + i of token t.
        if (t < T)
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {
                const int64_t o = o0 + 16 * rt + 4 * q;
                f32x4 y = c[rt];
#pragma unroll
                for (int e = 0; e < 4; ++e) y[e] += acc[rt][e];
                if (o < M) store_y4<YF32>(Y, t * ldy + o, M - o, yvec, y);
            }
    }
}

// ------------------------------------------------------------------ host

// K slices of z: enough workgroups (of 16 tokens and a slice) for every
// compute unit, at least 128 channels each, at most 32 partials to add.
static int64_t z_slices(int64_t T, int64_t K, int64_t* per) {
    const int64_t tiles = (T + 15) / 16;
    int64_t s = (512 + tiles - 1) / (tiles > 0 ? tiles : 1);
    const int64_t most = K / 128 > 0 ? K / 128 : 1;
    s = s > most ? most : s;
    s = s > 32 ? 32 : s < 1 ? 1 : s;
    *per = ((K + s - 1) / s + 31) / 32 * 32;
    return (K + *per - 1) / *per;
}

size_t adapters_ws_bytes(int64_t T, int64_t K, int rank) {
    int64_t per;
    return (size_t)z_slices(T, K, &per) * T * rank * 4;
}

template <bool XF32, bool AF32>
static hipError_t launch_z(const void* X, int64_t T, int64_t K, int64_t ldx, const AdapterTable& ad, float* Z,
                           hipStream_t st) {
    int64_t per;
    const int64_t s = z_slices(T, K, &per);
    const dim3 grid((unsigned)((T + 15) / 16), (unsigned)s);
#define TTQ_AZ(RT)                                                                                                     \
    return launch_kernel(k_adapter_z<XF32, AF32, RT>, grid, dim3(kAzWaves * kWave), 0, st, nullptr, nullptr, X, T, K, \
                         ldx, ad, per, Z)
    if (ad.rank <= 16) TTQ_AZ(1);
    if (ad.rank <= 32) TTQ_AZ(2);
    TTQ_AZ(4);
#undef TTQ_AZ
}

template <bool CF32, bool BF32, bool YF32>
static hipError_t launch_y(const float* Z, int64_t T, int64_t K, const AdapterTable& ad, const void* C, int64_t ldc,
                           int64_t M, void* Y, int64_t ldy, hipStream_t st) {
    int64_t per;
    const int s = (int)z_slices(T, K, &per);
    auto vec = [](const void* p, int64_t ld, bool f32) { return (uintptr_t)p % (f32 ? 16 : 8) == 0 && ld % 4 == 0; };
    const int cv = C != nullptr && vec(C, ldc, CF32), yv = vec(Y, ldy, YF32);
    const int64_t tiles = (T + 15) / 16;
#define TTQ_AY3(VEC, RT, ST)                                                                                          \
    do {                                                                                                              \
        const int64_t rb = (M + 16 * RT * kAyWaves - 1) / (16 * RT * kAyWaves);                                       \
        int64_t blocks = rb * tiles / 2048;                                                                           \
        blocks = blocks < 1 ? 1 : blocks > rb ? rb : blocks;                                                          \
        if ((rb + blocks - 1) / blocks > 65535) blocks = (rb + 65534) / 65535;                                        \
        return launch_kernel(k_adapter_y<CF32, BF32, YF32, VEC, RT, ST>,                                              \
                             dim3((unsigned)tiles, (unsigned)((rb + blocks - 1) / blocks)), dim3(kAyWaves * kWave),   \
                             0, st, nullptr, nullptr, Z, s, T, ad, C, ldc, M, Y, ldy, (int)blocks, cv, yv);           \
    } while (0)
#define TTQ_AY2(VEC, RT)                 \
    do {                                 \
        if (ad.rank <= 32) TTQ_AY3(VEC, RT, 1); \
        TTQ_AY3(VEC, RT, 2);             \
    } while (0)
    if (ad.rank % 8 != 0) TTQ_AY2(false, 1);
    if (T < 128) TTQ_AY2(true, 1);
    TTQ_AY2(true, 4);
#undef TTQ_AY2
#undef TTQ_AY3
}

hipError_t launch_adapters(const void* X, bool xf32, int64_t T, int64_t K, int64_t ldx, const AdapterTable& ad,
                           const void* C, bool cf32, int64_t ldc, int64_t M, void* Y, bool yf32, int64_t ldy, float* Z,
                           hipStream_t st) {
    hipError_t e;
    if (xf32) e = ad.f32 ? launch_z<true, true>(X, T, K, ldx, ad, Z, st) : launch_z<true, false>(X, T, K, ldx, ad, Z, st);
    else e = ad.f32 ? launch_z<false, true>(X, T, K, ldx, ad, Z, st) : launch_z<false, false>(X, T, K, ldx, ad, Z, st);
    if (e != hipSuccess) return e;
#define TTQ_AY(CF, YF)                                                                        \
    return ad.f32 ? launch_y<CF, true, YF>(Z, T, K, ad, C, ldc, M, Y, ldy, st)                \
                  : launch_y<CF, false, YF>(Z, T, K, ad, C, ldc, M, Y, ldy, st)
    if (cf32) {
        if (yf32) TTQ_AY(true, true);
        TTQ_AY(true, false);
    }
    if (yf32) TTQ_AY(false, true);
    TTQ_AY(false, false);
#undef TTQ_AY
}

}  // namespace ttq
