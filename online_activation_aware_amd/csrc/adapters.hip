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

// From here on the kernels for runs of one adapter: the ids lie on the device,
// so the number of tokens decides.  Runs of 100 tokens (in brackets an adapter of
// 64 for every token), bf16, rank 16 and 64, 4096 -> 4096, the kernels for few
// tokens against these: 128 tokens 11 (18) against 10 (61) us and 15 (30)
// against 15 (134); 256: 13 (29) / 12 (73), 20 (51) / 18 (138); 512: 26 (49) / 21
// (70), 42 (91) / 38 (135); 1024: 33 (84) / 20 (72), 54 (160) / 34 (143).  4096 ->
// 14336, rank 32, 256 adapters: 128 tokens 18 (35) / 11 (97), 256 28 (62) / 14 (103).
constexpr int64_t kRunsMinT = 512;

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
    const int r16 = threadIdx.x & 15;
    int first = r16;                              // the first token of this token's adapter
#pragma unroll
    for (int s = 1; s < 16; ++s) {
        const int other = __shfl(id, (r16 - s) & 15);
        if (s <= r16 && other == id) first = r16 - s;
    }
    const uint32_t lead = (uint32_t)__ballot(rk > 0 && first == r16) & 0xFFFFu;
    const int place = rk > 0 ? __builtin_popcount(lead & ((1u << first) - 1)) : -1;
    if (threadIdx.x < 16) {
        dof[r16] = place;
        if ((lead >> r16) & 1u) {
            dist[place] = id;
            dr[place] = rk;
        }
    }
    return __builtin_popcount(lead);
}

// ------------------------------------------------------------------ z

// A workgroup owns 16 tokens, one K slice and a share (grid.z) of the tile's
// distinct adapters; its items (adapter d, part c of the slice) go to the
// waves, several parts per adapter so that few adapters still use all of
// them.  RT: 16-row tiles of the rank.
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
    const int ng = (nd + (int)gridDim.z - 1) / (int)gridDim.z;       // adapters of this share
    const int dbeg = (int)blockIdx.z * ng, dn = min(ng, nd - dbeg);
    if (dn <= 0) return;
    const int parts = kAzWaves / dn > 0 ? kAzWaves / dn : 1;
    const int64_t steps = (k1 - k0 + 31) / 32, sp = (steps + parts - 1) / parts;
    const rsrc_t rx = make_rsrc((const char*)X + t0 * ldx * XE, ((rows - 1) * ldx + K) * XE);
    const int R = ad.rank;
    // Items in rounds of one per wave; after a round its adapters' sums go out.
    for (int base = 0; base < dn * parts; base += kAzWaves) {
        const int item = base + wave, d = dbeg + item / parts, c = item % parts;
        f32x4 acc[RT];
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) acc[rt] = f32x4{0.f, 0.f, 0.f, 0.f};
        if (item < dn * parts) {
            const int a = __builtin_amdgcn_readfirstlane(dist[d]);
            const int ra = __builtin_amdgcn_readfirstlane(dr[d]);
            const rsrc_t rA = make_rsrc((const char*)ad.A + (int64_t)a * R * K * AE, (int64_t)ra * K * AE);
            const int64_t sb = c * sp, se = min(steps, sb + sp);
            constexpr int U = XF32 || AF32 ? 2 : RT <= 2 ? 8 : 4;   // steps whose loads are in flight together
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
            const int d0 = dbeg + base / parts, pl = dof[r16];
            if (pl >= d0 && pl < min(d0 + kAzWaves / parts, dbeg + dn)) {
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

// kRunsMinT tokens or more, bf16 operands: a workgroup owns 32 tokens and one K
// slice and passes it 256 channels at a time through LDS, so that memory is
// read in rows of 512 consecutive bytes (the fragments above take 64 of each
// row, rows 2 K bytes apart: a power of two for most K) and a row of A serves
// both token tiles.  The next channels are in registers while one step is
// multiplied; wave w has channels 32 w ..+31 of each step, the waves' tiles are
// added in wave order.  One pass per distinct adapter, mostly one.
constexpr int kArzCh = 256;
constexpr int kArzRow = kArzCh * 2 + 16;          // LDS bytes of a row, 16 apart modulo the banks

template <int RT>
__global__ __launch_bounds__(kAzWaves * kWave) void k_adapter_z_runs(const uint16_t* __restrict__ X, int64_t T,
                                                                     int64_t K, int64_t ldx, AdapterTable ad,
                                                                     int64_t per, float* __restrict__ Z) {
    constexpr int kTok = 32;
    constexpr int NP = (kTok + 16 * RT) * (kArzCh / 8) / (kAzWaves * kWave);   // 16-byte pieces a thread stages
    constexpr int kTile = (kTok + 16 * RT) * kArzRow, kRed = kAzWaves * 2 * RT * kWave * 16;
    __shared__ __attribute__((aligned(16))) unsigned char smem[kTile > kRed ? kTile : kRed];
    const int tid = threadIdx.x, lane = tid & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int r16 = lane & 15, q = lane >> 4;
    const int64_t t0 = (int64_t)blockIdx.x * kTok;
    const int64_t k0 = (int64_t)blockIdx.y * per, k1 = min(K, k0 + per);
    const int64_t rows = min((int64_t)kTok, T - t0);
    const int R = ad.rank;
    const int id = (lane & 31) < rows ? ad.ids[t0 + (lane & 31)] : -1;   // lanes 0..31 and again 32..63
    const int rk = adapter_rank(ad, id);
    const rsrc_t rx = make_rsrc(X + t0 * ldx, ((rows - 1) * ldx + K) * 2);
    uint32_t left = (uint32_t)__ballot(rk > 0);
    while (left) {                                // at most 32 rounds: each takes its first token's bit
        const int f = __builtin_ctz(left);
        const int a = __builtin_amdgcn_readlane(id, f), ra = __builtin_amdgcn_readlane(rk, f);
        const bool mine = rk > 0 && id == a;
        left &= ~(uint32_t)__ballot(mine);
        const rsrc_t rA = make_rsrc((const uint16_t*)ad.A + (int64_t)a * R * K, (int64_t)ra * K * 2);
        u32x4 v[NP];
        auto fetch = [&](int64_t k) __attribute__((always_inline)) {
#pragma unroll
            for (int n = 0; n < NP; ++n) {
                const int p = tid + n * kAzWaves * kWave, r = p / (kArzCh / 8);
                const int64_t j = k + p % (kArzCh / 8) * 8;   // K % 8 == 0: all in or all out
                const uint32_t off = j >= k1 ? kOut : (uint32_t)((r < kTok ? r * ldx : (r - kTok) * K) + j) * 2;
                // A wave's pieces are of X or of A alone.
                v[n] = __builtin_bit_cast(u32x4, r < kTok ? __builtin_amdgcn_raw_buffer_load_b128(rx, (int)(r < rows ? off : kOut), 0, 0)
                                                          : __builtin_amdgcn_raw_buffer_load_b128(rA, (int)off, 0, 0));
            }
        };
        f32x4 acc[2][RT];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) acc[h][rt] = f32x4{0.f, 0.f, 0.f, 0.f};
        fetch(k0);
        for (int64_t k = k0; k < k1; k += kArzCh) {
            __syncthreads();                      // what was there has been read
#pragma unroll
            for (int n = 0; n < NP; ++n) {
                const int p = tid + n * kAzWaves * kWave;
                *(u32x4*)(smem + p / (kArzCh / 8) * kArzRow + p % (kArzCh / 8) * 16) = v[n];
            }
            if (k + kArzCh < k1) fetch(k + kArzCh);
            sync_lds();
            const unsigned char* b = smem + 64 * wave + 16 * q + r16 * kArzRow;
            u32x4 x[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) x[h] = *(const u32x4*)(b + 16 * h * kArzRow);
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {
                const u32x4 w = *(const u32x4*)(b + (kTok + 16 * rt) * kArzRow);
#pragma unroll
                for (int h = 0; h < 2; ++h) acc[h][rt] = mfma_16x16x32(w, x[h], acc[h][rt]);
            }
        }
        __syncthreads();
        f32x4* red = (f32x4*)smem;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) red[((wave * 2 + h) * RT + rt) * kWave + lane] = acc[h][rt];
        __syncthreads();
        // Lane of tile (h, rt): z^T[16 rt + 4 q + i][16 h + r16].
        for (int w = wave; w < 2 * RT; w += kAzWaves) {
            const int h = w / RT, rt = w % RT;
            const bool take = __shfl((int)mine, 16 * h + r16) != 0;
            f32x4 z = red[w * kWave + lane];
            for (int u = 1; u < kAzWaves; ++u) {
                const f32x4 y = red[(u * 2 * RT + w) * kWave + lane];
#pragma unroll
                for (int i = 0; i < 4; ++i) z[i] += y[i];
            }
            if (take)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int kk = 16 * rt + 4 * q + i;
                    if (kk < R) Z[((int64_t)blockIdx.y * T + t0 + 16 * h + r16) * R + kk] = z[i];
                }
        }
    }
}

// ------------------------------------------------------------------ Y

// Few tokens (or odd sizes): a wave owns 16 tokens and 16 rows of M at a time;
// workgroup: 4 waves on the same tokens.  Its items, batches of U adapters,
// are loaded one ahead (the first before z is summed).  VEC: R % 8 == 0.
// ST: 32-slot steps of the rank.  C comes as `cparts` fp32 partial sums where
// it is a projection split over K, added in order.
constexpr int kAyWaves = 4;

// Four consecutive values of C as loaded: fp32 bits, or bf16 pairs in the
// first two words.
template <bool CF32>
__device__ __forceinline__ u32x4 load_c4(const void* C, int64_t i, int64_t avail, bool vec) {
    u32x4 v = u32x4{0u, 0u, 0u, 0u};
    if (vec && avail >= 4) {
        if constexpr (CF32) return *(const u32x4*)((const uint32_t*)C + i);
        const u32x2 c = *(const u32x2*)((const uint16_t*)C + i);
        return u32x4{c[0], c[1], 0u, 0u};
    }
#pragma unroll
    for (int r = 0; r < 4; ++r)
        if (r < avail) {
            if constexpr (CF32) v[r] = ((const uint32_t*)C)[i + r];
            else v[r / 2] |= (uint32_t)((const uint16_t*)C)[i + r] << (16 * (r & 1));
        }
    return v;
}
template <bool CF32>
__device__ __forceinline__ f32x4 c4_values(const u32x4& c) {
    if constexpr (CF32) return __builtin_bit_cast(f32x4, c);
    else return f32x4{bf16lo_to_f32(c[0]), bf16hi_to_f32(c[0]), bf16lo_to_f32(c[1]), bf16hi_to_f32(c[1])};
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

template <bool CF32, bool BF32, bool YF32, bool VEC, int ST>
__global__ __launch_bounds__(kAyWaves * kWave) void k_adapter_y(const float* __restrict__ Z, int slices, int64_t T,
                                                                AdapterTable ad, ProjectionIn ci, int64_t M, void* Y,
                                                                int64_t ldy, int blocks, int share, int cvec,
                                                                int yvec) {
    constexpr int BE = BF32 ? 4 : 2;
    constexpr int U = 8;
    constexpr int kZRow = 32 * ST + 4;
    constexpr int kZn = 32 * ST * 16 / (kAyWaves * kWave);   // z values a thread sums
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
    // share: the waves on one row tile, wave j of them with the tile's adapters
    // j, j + share, ... (1, or all four where rows alone leave the chip idle).
    const int dw = wave % share, mine_n = nd > dw ? (nd - dw + share - 1) / share : 0;
    const int batches = mine_n == 0 ? 1 : (mine_n + U - 1) / U;
    const int64_t wb0 = (int64_t)blockIdx.y * blocks;        // row blocks of 16 rows per wave on its own
    auto row0 = [&](int bi) -> int64_t { return ((wb0 + bi) * (kAyWaves / share) + wave / share) * 16; };
    int nblk = 0;                                 // blocks this wave has rows in
    while (nblk < blocks && row0(nblk) < M) ++nblk;
    const int items = nblk * batches;
    sync_lds();                                   // dist, dr, dof

    // z of the tile, slices in order, times the adapters' scales: the tile's
    // 16 R values are consecutive.
    float zv[kZn];
    int zt[kZn], zk[kZn];
#pragma unroll
    for (int n = 0; n < kZn; ++n) {
        const int i = tid + n * kAyWaves * kWave;
        zt[n] = i / R;
        zk[n] = i - zt[n] * R;
        zv[n] = 0.f;
    }
    const float sl = rk > 0 && ad.scale != nullptr ? ad.scale[id] : 1.f;
    const int64_t zstep = T * R;
    const float* zp = Z + t0 * R + tid;
    for (int i0 = 0; i0 < slices; i0 += 4) {
        float x[kZn][4];
#pragma unroll
        for (int n = 0; n < kZn; ++n)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                x[n][j] = zt[n] < 16 && t0 + zt[n] < T && i0 + j < slices
                              ? zp[(i0 + j) * zstep + n * kAyWaves * kWave] : 0.f;
#pragma unroll
        for (int n = 0; n < kZn; ++n)
#pragma unroll
            for (int j = 0; j < 4; ++j) zv[n] += x[n][j];
    }

    constexpr int kParts = CF32 ? 4 : 1;          // partial sums of C loaded ahead
    struct Item {
        Eight<BF32> b[U][ST];
        u32x4 c[kParts];
    };
    const int place = dof[r16];
    // Tokens whose outputs this wave writes.
    const bool own = t < T && (place >= 0 ? place % share == dw : dw == 0);
    auto load = [&](Item& it, int i) __attribute__((always_inline)) {
        const int bi = i / batches, d0 = (i - bi * batches) * U;
        const int64_t o0 = row0(bi), o = o0 + 4 * q;
        if (d0 == 0 && ci.C != nullptr)
#pragma unroll
            for (int p = 0; p < kParts; ++p)
                if (p < ci.parts) {
                    const char* c = (const char*)ci.C + p * ci.stride * 4;
                    it.c[p] = load_c4<CF32>(c, t * ci.ldc + o, own ? M - o : 0, cvec);
                }
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (d0 + u < mine_n) {                // uniform
                const int d = dw + (d0 + u) * share;
                const int a = __builtin_amdgcn_readfirstlane(dist[d]);
                const int ra = __builtin_amdgcn_readfirstlane(dr[d]);
                const rsrc_t rB = make_rsrc((const char*)ad.B + ((int64_t)a * M + o0) * R * BE,
                                            min((int64_t)16, M - o0) * R * BE);
#pragma unroll
                for (int s = 0; s < ST; ++s)
                    it.b[u][s] = load_b<BF32, VEC>(rB, r16, 32 * s + 8 * q, ra, R, o0 + r16 < M);
            }
    };
    Item i0, i1;
    if (items > 0) load(i0, 0);
#pragma unroll
    for (int n = 0; n < kZn; ++n) {
        const int zr = __shfl(rk, zt[n] & 15);    // lanes 0..15 of every wave hold the tokens
        const float sc = __shfl(sl, zt[n] & 15);
        if (zt[n] < 16) zl[zt[n]][zk[n]] = zk[n] < zr ? zv[n] * sc : 0.f;
    }
    sync_lds();
    ZOp<BF32> zo[ST];
#pragma unroll
    for (int s = 0; s < ST; ++s) {
        float z[8];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const f32x4 v = *(const f32x4*)&zl[r16][32 * s + 8 * q + 4 * h];
#pragma unroll
            for (int e = 0; e < 4; ++e) z[4 * h + e] = 32 * s + 8 * q + 4 * h + e < rk ? v[e] : 0.f;
        }
        zo[s] = z_operand<BF32>(z);
    }
    f32x4 acc, c;
    auto compute = [&](const Item& it, int i) __attribute__((always_inline)) {
        const int bi = i / batches, d0 = (i - bi * batches) * U;
        const int64_t o = row0(bi) + 4 * q;
        if (d0 == 0) {
            acc = c = f32x4{0.f, 0.f, 0.f, 0.f};
            if (ci.C != nullptr) {
                c = c4_values<CF32>(it.c[0]);
                if constexpr (CF32) {
#pragma unroll
                    for (int p = 1; p < kParts; ++p)
                        if (p < ci.parts) {
                            const f32x4 v = c4_values<true>(it.c[p]);
#pragma unroll
                            for (int e = 0; e < 4; ++e) c[e] += v[e];
                        }
                    for (int p = kParts; p < ci.parts; ++p) {
                        const f32x4 v = c4_values<true>(
                            load_c4<true>((const float*)ci.C + p * ci.stride, t * ci.ldc + o, own ? M - o : 0, cvec));
#pragma unroll
                        for (int e = 0; e < 4; ++e) c[e] += v[e];
                    }
                }
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (d0 + u < mine_n) {
                const bool mine = place == dw + (d0 + u) * share;
                f32x4 p = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int s = 0; s < ST; ++s) p = mac_z<BF32>(it.b[u][s], zo[s], p);
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[e] = mine ? p[e] : acc[e];
            }
        // Lane: rows 4 q + e of token t.
        if (d0 + U >= mine_n && own && o < M) {
#pragma unroll
            for (int e = 0; e < 4; ++e) c[e] += acc[e];
            store_y4<YF32>(Y, t * ldy + o, M - o, yvec, c);
        }
    };
    for (int i = 0; i < items; i += 2) {
        if (i + 1 < items) load(i1, i + 1);
        __builtin_amdgcn_sched_barrier(0);
        compute(i0, i);
        if (i + 1 >= items) break;
        if (i + 2 < items) load(i0, i + 2);
        __builtin_amdgcn_sched_barrier(0);
        compute(i1, i + 1);
    }
}

// One token: a single launch.  Every workgroup (128 rows of M, four threads a
// row) forms z itself, a wave a rank at a time; A passes through the L2 once
// per workgroup, which for small A costs less than a second launch (4096 ->
// 4096, rank 16: 5.0 us, 9.4 us in two).
constexpr int kA1Rows = 128, kA1Threads = 512;
constexpr int64_t kA1Bytes = (int64_t)16 << 20;   // of A over all workgroups

template <bool XF32, bool AF32, bool CF32, bool YF32>
__global__ __launch_bounds__(kA1Threads) void k_adapter_one(const void* __restrict__ X, int64_t K, AdapterTable ad,
                                                            ProjectionIn ci, int64_t M, void* Y) {
    __shared__ float z[64];
    constexpr int XE = XF32 ? 4 : 2, AE = AF32 ? 4 : 2;
    const int tid = threadIdx.x, lane = tid & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int a = __builtin_amdgcn_readfirstlane(ad.ids[0]);
    const int ra = __builtin_amdgcn_readfirstlane(adapter_rank(ad, a));
    const int R = ad.rank;
    const int64_t o = (int64_t)blockIdx.x * kA1Rows + tid / 4;
    const rsrc_t rx = make_rsrc(X, K * XE);
    constexpr int U = 4;                          // pieces of 8 channels in flight
    for (int k = wave; k < ra; k += kA1Threads / kWave) {
        const rsrc_t rA = make_rsrc((const char*)ad.A + ((int64_t)a * R + k) * K * AE, K * AE);
        float s = 0.f;
        for (int64_t j0 = 8 * lane; j0 < K; j0 += 8 * U * kWave) {
            Eight<XF32> x[U];
            Eight<AF32> w[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {         // behind K: zeros
                x[u] = load_eight<XF32>(rx, (uint32_t)((j0 + 8 * u * kWave) * XE));
                w[u] = load_eight<AF32>(rA, (uint32_t)((j0 + 8 * u * kWave) * AE));
            }
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int e = 0; e < 8; ++e) s = __builtin_fmaf(eight_at<AF32>(w[u], e), eight_at<XF32>(x[u], e), s);
        }
#pragma unroll
        for (int m = 1; m < kWave; m <<= 1) s += __shfl_xor(s, m);
        if (lane == 0) z[k] = s;
    }
    __syncthreads();
    if (o >= M) return;                           // whole quads
    float y = 0.f;
    for (int k = tid & 3; k < ra; k += 4) {
        const int64_t i = ((int64_t)a * M + o) * R + k;
        y = __builtin_fmaf(AF32 ? ((const float*)ad.B)[i] : bf16_to_f32(((const uint16_t*)ad.B)[i]), z[k], y);
    }
    y += __shfl_xor(y, 1);
    y += __shfl_xor(y, 2);
    if ((tid & 3) != 0) return;
    if (ra > 0 && ad.scale != nullptr) y *= ad.scale[a];
    float c = 0.f;
    if (ci.C != nullptr) c = CF32 ? ((const float*)ci.C)[o] : bf16_to_f32(((const uint16_t*)ci.C)[o]);
    if (ra > 0) c += y;
    if constexpr (YF32) ((float*)Y)[o] = c;
    else ((uint16_t*)Y)[o] = (uint16_t)f32_to_bf16(c);
}

// kRunsMinT tokens or more, mostly runs of one adapter: a wave owns 64 rows of M,
// keeps their B in registers and goes through four tiles of 16 tokens, all of
// whose C it has requested at the start; a tile of several adapters, or another one
// than the last, loads its B.  Column m of row tile rt is row 16 (m / 4) +
// 4 rt + m % 4 of the 64, so that a lane ends with 16 consecutive outputs of
// one token.  R, M and the strides multiples of 8, 16-byte aligned C and Y.
constexpr int kArTiles = 4;

template <bool CF32, bool BF32, bool YF32, int ST>
__global__ __launch_bounds__(kAyWaves * kWave) void k_adapter_runs(const float* __restrict__ Z, int slices, int64_t T,
                                                                   AdapterTable ad, ProjectionIn ci, int64_t M, void* Y,
                                                                   int64_t ldy) {
    constexpr int BE = BF32 ? 4 : 2;
    constexpr int CW = CF32 ? 4 : 2;              // 16-byte pieces of 16 values
    constexpr int kTok = 16 * kArTiles;
    constexpr int kZp = kTok * 8 * ST / (kAyWaves * kWave);   // 16-byte pieces of z a thread sums
    static_assert(kTok == kWave, "a lane per token");
    __shared__ __attribute__((aligned(16))) float zl[kTok][32 * ST + 4];
    const int tid = threadIdx.x, lane = tid & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int r16 = lane & 15, q = lane >> 4;
    const int64_t tb = (int64_t)blockIdx.y * kTok;
    const int64_t o0 = ((int64_t)blockIdx.x * kAyWaves + wave) * 64;
    const int R = ad.rank;
    const int64_t mrows = min((int64_t)64, M - o0);
    // Lane l: token tb + l of the four tiles.
    const int id_l = tb + lane < T ? ad.ids[tb + lane] : -1;
    const int rk_l = adapter_rank(ad, id_l);
    const float sc_l = rk_l > 0 && ad.scale != nullptr ? ad.scale[id_l] : 1.f;

    // z of the 64 tokens, slices in order, once for the four waves; requested
    // before everything else, then C of the four tiles and B of the first
    // adapter.
    const int per = R / 4;                        // 16-byte pieces of a row of z
    // Slices whose loads are in flight together (one after the other: 2048 tokens,
    // 4096 -> 4096, rank 64, 32.7 us; four 30.4, two, with fewer registers, 30.1).
    constexpr int kZs = ST == 1 ? 4 : 2;
    f32x4 zv[kZs][kZp];
    const int64_t have = min((int64_t)kTok, T - tb) * per;
    auto load_z = [&](int p0) __attribute__((always_inline)) {
#pragma unroll
        for (int p = 0; p < kZs; ++p) {
            const rsrc_t rz = make_rsrc(Z + ((int64_t)(p0 + p) * T + tb) * R, p0 + p < slices ? have * 16 : 0);
#pragma unroll
            for (int n = 0; n < kZp; ++n)         // behind the tokens or slices: zeros
                zv[p][n] = __builtin_bit_cast(
                    f32x4, __builtin_amdgcn_raw_buffer_load_b128(rz, (tid + n * kAyWaves * kWave) * 16, 0, 0));
        }
    };
    load_z(0);
    const bool oin = o0 + 16 * q < M;             // 16 consecutive rows, in eights
    u32x4 c[kArTiles][CW];
#pragma unroll
    for (int i = 0; i < kArTiles; ++i) {
        const int64_t t = tb + 16 * i + r16;
        const char* cp = (const char*)ci.C + (t * ci.ldc + o0 + 16 * q) * (CF32 ? 4 : 2);
#pragma unroll
        for (int w = 0; w < CW; ++w)
            if (ci.C != nullptr && t < T && o0 + 16 * q + w * (CF32 ? 4 : 8) < M) c[i][w] = *(const u32x4*)(cp + 16 * w);
    }
    int cur = -1;                                 // the adapter whose B is held
    Eight<BF32> b[4][ST];
    auto load_rows = [&](int a, int ra) __attribute__((always_inline)) {
        cur = a;
        const rsrc_t rB = make_rsrc((const char*)ad.B + ((int64_t)a * M + o0) * R * BE, mrows * R * BE);
#pragma unroll
        for (int rt = 0; rt < 4; ++rt)
#pragma unroll
            for (int h = 0; h < ST; ++h) {
                const int r = 16 * (r16 >> 2) + 4 * rt + (r16 & 3);
                b[rt][h] = load_b<BF32, true>(rB, r, 32 * h + 8 * q, ra, R, r < mrows);
            }
    };
    if (const uint64_t any = __ballot(rk_l > 0); any != 0 && o0 < M) {
        const int f = __builtin_ctzll(any);
        load_rows(__builtin_amdgcn_readlane(id_l, f), __builtin_amdgcn_readlane(rk_l, f));
    }
    f32x4 zs[kZp];
#pragma unroll
    for (int n = 0; n < kZp; ++n) zs[n] = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int p0 = 0;;) {
#pragma unroll
        for (int p = 0; p < kZs; ++p)
#pragma unroll
            for (int n = 0; n < kZp; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) zs[n][e] += zv[p][n][e];
        p0 += kZs;
        if (p0 >= slices) break;
        load_z(p0);
    }
#pragma unroll
    for (int n = 0; n < kZp; ++n) {               // times the adapters' scales
        const int i = tid + n * kAyWaves * kWave, t = i / per, k = (i - t * per) * 4;
        const float sc = __shfl(sc_l, t & (kWave - 1));
        if (t < kTok) {
#pragma unroll
            for (int e = 0; e < 4; ++e) zl[t][k + e] = zs[n][e] * sc;
        }
    }
    sync_lds();
    if (o0 >= M) return;
    auto compute = [&](int i) __attribute__((always_inline)) {
        const int id = __shfl(id_l, 16 * i + r16), rk = __shfl(rk_l, 16 * i + r16);
        ZOp<BF32> zo[ST];
#pragma unroll
        for (int h = 0; h < ST; ++h) {
            f32x4 v[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) v[e] = *(const f32x4*)&zl[16 * i + r16][32 * h + 8 * q + 4 * e];
            float z[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) z[e] = 32 * h + 8 * q + e < rk ? v[e / 4][e % 4] : 0.f;
            zo[h] = z_operand<BF32>(z);
        }
        f32x4 acc[4];
#pragma unroll
        for (int rt = 0; rt < 4; ++rt) acc[rt] = f32x4{0.f, 0.f, 0.f, 0.f};
        uint32_t left = (uint32_t)__ballot(rk > 0) & 0xFFFFu;
        while (left) {                            // at most 16 rounds
            const int f = __builtin_ctz(left);
            const int a = __builtin_amdgcn_readlane(id, f);
            const bool mine = rk > 0 && id == a;
            left &= ~((uint32_t)__ballot(mine) & 0xFFFFu);
            if (a != cur) load_rows(a, __builtin_amdgcn_readlane(rk, f));   // uniform
#pragma unroll
            for (int rt = 0; rt < 4; ++rt) {
                f32x4 p = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int h = 0; h < ST; ++h) p = mac_z<BF32>(b[rt][h], zo[h], p);
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[rt][e] = mine ? p[e] : acc[rt][e];
            }
        }
        // Lane: rows 16 q + 4 rt + e of token t.
        const int64_t t = tb + 16 * i + r16;
        if (t >= T || !oin) return;
        if (ci.C != nullptr)
#pragma unroll
            for (int rt = 0; rt < 4; ++rt) {
                f32x4 v;
                if constexpr (CF32) v = c4_values<true>(c[i][rt]);
                else v = c4_values<false>(u32x4{c[i][rt / 2][2 * (rt & 1)], c[i][rt / 2][2 * (rt & 1) + 1], 0u, 0u});
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[rt][e] += v[e];
            }
        const int64_t o = o0 + 16 * q;
        if constexpr (YF32) {
#pragma unroll
            for (int rt = 0; rt < 4; ++rt)
                if (o + 4 * rt < M) *(f32x4*)((float*)Y + t * ldy + o + 4 * rt) = acc[rt];
        } else {
#pragma unroll
            for (int h = 0; h < 2; ++h)
                if (o + 8 * h < M)
                    *(u32x4*)((uint16_t*)Y + t * ldy + o + 8 * h) =
                        u32x4{pack_bf16x2(acc[2 * h][0], acc[2 * h][1]), pack_bf16x2(acc[2 * h][2], acc[2 * h][3]),
                              pack_bf16x2(acc[2 * h + 1][0], acc[2 * h + 1][1]),
                              pack_bf16x2(acc[2 * h + 1][2], acc[2 * h + 1][3])};
        }
    };
#pragma unroll
    for (int i = 0; i < kArTiles; ++i) {
        compute(i);
        __builtin_amdgcn_sched_barrier(0);
    }
}

// ------------------------------------------------------------------ host

// K slices of z, whose partials every workgroup of the second launch adds:
// at most eight, of at least 512 channels.  A tile of a few requests spreads
// over the chip by its adapters as well (sixteen shares), its slices are of at
// least 1024 (48 requests: 22.8 us; eight shares 23.9, slices of 512 24.5);
// kRunsMinT tokens or more (runs of few adapters) by their tiles.
static int z_shares(int64_t T) { return T == 1 || T >= kRunsMinT ? 1 : 16; }
static int64_t z_slices(int64_t T, int64_t K, int64_t* per) {
    const int64_t tiles = (T + 15) / 16;
    int64_t s = tiles > 0 ? (T < kRunsMinT ? 8 : (512 + tiles - 1) / tiles) : 1;
    const int64_t least = T > 1 && T < kRunsMinT ? 1024 : 512, most = K / least > 0 ? K / least : 1;
    s = s > most ? most : s;
    s = s > 8 ? 8 : s;
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
    if constexpr (!XF32 && !AF32)
        if (T >= kRunsMinT) {
            const dim3 grid((unsigned)((T + 31) / 32), (unsigned)s);
#define TTQ_AZR(RT)                                                                                                  \
    return launch_kernel(k_adapter_z_runs<RT>, grid, dim3(kAzWaves * kWave), 0, st, nullptr, nullptr,                \
                         (const uint16_t*)X, T, K, ldx, ad, per, Z)
            if (ad.rank <= 16) TTQ_AZR(1);
            if (ad.rank <= 32) TTQ_AZR(2);
            TTQ_AZR(4);
#undef TTQ_AZR
        }
    const dim3 grid((unsigned)((T + 15) / 16), (unsigned)s, (unsigned)z_shares(T));
#define TTQ_AZ(RT)                                                                                                     \
    return launch_kernel(k_adapter_z<XF32, AF32, RT>, grid, dim3(kAzWaves * kWave), 0, st, nullptr, nullptr, X, T, K, \
                         ldx, ad, per, Z)
    if (ad.rank <= 16) TTQ_AZ(1);
    if (ad.rank <= 32) TTQ_AZ(2);
    TTQ_AZ(4);
#undef TTQ_AZ
}

template <bool CF32, bool BF32, bool YF32>
static hipError_t launch_y(const float* Z, int64_t T, int64_t K, const AdapterTable& ad, const ProjectionIn& ci,
                           int64_t M, void* Y, int64_t ldy, hipStream_t st) {
    int64_t per;
    const int s = (int)z_slices(T, K, &per);
    // Rows of four values (the vector accesses of k_adapter_y), and what
    // k_adapter_runs needs.
    auto vec = [](const void* p, int64_t ld, bool f32) { return (uintptr_t)p % (f32 ? 16 : 8) == 0 && ld % 4 == 0; };
    auto vec16 = [](const void* p, int64_t ld) { return (uintptr_t)p % 16 == 0 && ld % 8 == 0; };
    const int cv = ci.C != nullptr && vec(ci.C, ci.ldc, CF32) && ci.stride % 4 == 0, yv = vec(Y, ldy, YF32);
    if (T >= kRunsMinT && ad.rank % 8 == 0 && M % 8 == 0 && vec16(Y, ldy) && ci.parts == 1 &&
        (ci.C == nullptr || vec16(ci.C, ci.ldc))) {
        const dim3 grid((unsigned)((M + 64 * kAyWaves - 1) / (64 * kAyWaves)),
                        (unsigned)((T + 16 * kArTiles - 1) / (16 * kArTiles)));
        if (grid.y <= 65535)
            return ad.rank <= 32
                       ? launch_kernel(k_adapter_runs<CF32, BF32, YF32, 1>, grid, dim3(kAyWaves * kWave), 0, st, nullptr,
                                       nullptr, Z, s, T, ad, ci, M, Y, ldy)
                       : launch_kernel(k_adapter_runs<CF32, BF32, YF32, 2>, grid, dim3(kAyWaves * kWave), 0, st, nullptr,
                                       nullptr, Z, s, T, ad, ci, M, Y, ldy);
    }
    const int64_t tiles = (T + 15) / 16;
    // All four waves on one row tile while that gives fewer than four waves
    // per SIMD and there can be several adapters.
    const int share = T > 1 && tiles * ((M + 15) / 16) * kAyWaves <= 4096 ? kAyWaves : 1;
    const int64_t rows = 16 * (kAyWaves / share), rb = (M + rows - 1) / rows;
    int64_t blocks = rb * tiles / 2048;           // row blocks per workgroup, once the chip is full
    blocks = blocks < 1 ? 1 : blocks > rb ? rb : blocks;
    if ((rb + blocks - 1) / blocks > 65535) blocks = (rb + 65534) / 65535;
    const dim3 grid((unsigned)tiles, (unsigned)((rb + blocks - 1) / blocks));
#define TTQ_AY2(VEC, ST)                                                                                            \
    return launch_kernel(k_adapter_y<CF32, BF32, YF32, VEC, ST>, grid, dim3(kAyWaves * kWave), 0, st, nullptr,      \
                         nullptr, Z, s, T, ad, ci, M, Y, ldy, (int)blocks, share, cv, yv)
    if (ad.rank % 8 != 0) {
        if (ad.rank <= 32) TTQ_AY2(false, 1);
        TTQ_AY2(false, 2);
    }
    if (ad.rank <= 32) TTQ_AY2(true, 1);
    TTQ_AY2(true, 2);
#undef TTQ_AY2
}

template <bool CF32, bool YF32>
static hipError_t launch_one(const void* X, bool xf32, int64_t K, const AdapterTable& ad, const ProjectionIn& ci, int64_t M,
                             void* Y, hipStream_t st) {
    const dim3 grid((unsigned)((M + kA1Rows - 1) / kA1Rows)), block(kA1Threads);
#define TTQ_A1(XF, AF) \
    return launch_kernel(k_adapter_one<XF, AF, CF32, YF32>, grid, block, 0, st, nullptr, nullptr, X, K, ad, ci, M, Y)
    if (xf32) {
        if (ad.f32) TTQ_A1(true, true);
        TTQ_A1(true, false);
    }
    if (ad.f32) TTQ_A1(false, true);
    TTQ_A1(false, false);
#undef TTQ_A1
}

// C has Y's dtype or fp32.
hipError_t launch_adapters(const void* X, bool xf32, int64_t T, int64_t K, int64_t ldx, const AdapterTable& ad,
                           const ProjectionIn& ci, int64_t M, void* Y, bool yf32, int64_t ldy, float* Z,
                           hipStream_t st) {
    // (Not where Y lies on X: its first workgroups would write over what the
    // last still read.)
    const char *x0 = (const char*)X, *y0 = (const char*)Y;
    const bool apart = x0 + K * (xf32 ? 4 : 2) <= y0 || y0 + M * (yf32 ? 4 : 2) <= x0;
    if (T == 1 && ci.parts == 1 && apart &&
        (M + kA1Rows - 1) / kA1Rows * ad.rank * K * (ad.f32 ? 4 : 2) <= kA1Bytes) {
        if (yf32) return launch_one<true, true>(X, xf32, K, ad, ci, M, Y, st);
        return ci.f32 ? launch_one<true, false>(X, xf32, K, ad, ci, M, Y, st)
                      : launch_one<false, false>(X, xf32, K, ad, ci, M, Y, st);
    }
    hipError_t e;
    if (xf32) e = ad.f32 ? launch_z<true, true>(X, T, K, ldx, ad, Z, st) : launch_z<true, false>(X, T, K, ldx, ad, Z, st);
    else e = ad.f32 ? launch_z<false, true>(X, T, K, ldx, ad, Z, st) : launch_z<false, false>(X, T, K, ldx, ad, Z, st);
    if (e != hipSuccess) return e;
#define TTQ_AY(CF, YF)                                                                 \
    return ad.f32 ? launch_y<CF, true, YF>(Z, T, K, ad, ci, M, Y, ldy, st)             \
                  : launch_y<CF, false, YF>(Z, T, K, ad, ci, M, Y, ldy, st)
    if (yf32) TTQ_AY(true, true);
    if (ci.f32) TTQ_AY(true, false);
    TTQ_AY(false, false);
#undef TTQ_AY
}

}  // namespace ttq
