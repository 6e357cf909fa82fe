// A gated mixture-of-experts layer, of long prompts too, in 8-bit integers:
//   Y[t] = sum_j w[t][j] D_e h^,  h = act(g) u / s_down,  [g; u] = G_e x^,
// x^ and h^ the rows of X / s_in and of h in 8 bits, e = ids[t][j].
//
// The slots are sorted by expert; the first product reads its rows of X through
// that order (a token is quantized once for all of its experts, where they
// share s_in, and no row is copied) and its epilogue leaves h in fp32: a row's
// scale needs the whole row, and a bf16 h would move one code in eight.  The
// rows of h in 8 bits go through the second product into fp32 rows, which are
// weighted and added per token.
#include <algorithm>

#include "i8.hpp"
#include "rows_i8.hpp"
#include "sort.hpp"

namespace ttq {

// Few slots: workgroup 0 sorts them while the others quantize the tokens' rows.
// (The layer for 64 tokens of 2048 channels, 6 experts each: 102.7 us with two launches, 98.3.)
template <bool F32>
__global__ __launch_bounds__(kSortThreads) void k_moe_sort_rows(SortArgs s, I8RowsArgs r) {
    if (blockIdx.x == 0) sort_block<true>(s, 0, 1);
    else quantize_rows<F32, 2, true>(r, blockIdx.x - 1, gridDim.x - 1);
}

struct MoeI8Layout {
    size_t offsets, order, pos, sort, q, qs, h, hq, hs, total;
};

// The second product's rows are 16-byte aligned.
static int64_t row_floats(int64_t M) { return (M + 3) / 4 * 4; }

static MoeI8Layout moe_i8_layout(int64_t T, int64_t topk, int64_t K, int64_t I, int64_t M, int64_t E) {
    auto up = [](size_t n) { return (n + 255) / 256 * 256; };
    const size_t n = (size_t)(T * topk);
    MoeI8Layout L{};
    L.offsets = 0;
    L.order = L.offsets + up((size_t)(E + 1) * 4);
    L.pos = L.order + up(n * 4);
    L.sort = L.pos + up(n * 4);
    L.q = L.sort + up(moe_sort_ws_bytes(T * topk, E));
    L.qs = L.q + up(n * K);
    L.hq = L.qs + up(n * 4);
    L.hs = L.hq + up(n * I);
    L.h = L.hs + up(n * 4);                       // h, and when it is quantized the second product's rows
    const int64_t mp = row_floats(M);
    L.total = L.h + up(n * (size_t)(I > mp ? I : mp) * 4);
    return L;
}

size_t moe_i8_ws_bytes(int64_t T, int64_t topk, int64_t K, int64_t I, int64_t M, int64_t E) {
    return moe_i8_layout(T, topk, K, I, M, E).total;
}

hipError_t launch_moe_i8(const ttq_moe_i8_args* a, char* ws, hipStream_t st) {
    const MoeI8Layout L = moe_i8_layout(a->T, a->topk, a->K, a->I, a->M, a->E);
    const int64_t n = a->T * a->topk;
    const int E = (int)a->E, topk = (int)a->topk;
    int32_t *offsets = (int32_t*)(ws + L.offsets), *order = (int32_t*)(ws + L.order), *pos = (int32_t*)(ws + L.pos);
    int8_t *q = (int8_t*)(ws + L.q), *hq = (int8_t*)(ws + L.hq);
    float *qs = (float*)(ws + L.qs), *hs = (float*)(ws + L.hs), *h = (float*)(ws + L.h);
    const bool per = a->gate_up.s_stride != 0;    // an s_in for each expert: rows of slots, sorted, else of tokens
    I8RowsArgs rq{a->X, a->xt == TTQ_F32, a->ldx, per ? n : a->T, a->K, a->gate_up.s, true, q, a->K, qs};
    hipError_t e;
    if (!per && n <= kSortAlone && a->K <= kSortThreads * kRowSeg * kRowSegs) {
        const SortArgs s = sort_args(a->ids, n, E, offsets, order, pos, nullptr);
        const dim3 grid((unsigned)std::min<int64_t>(a->T, 511) + 1), block(kSortThreads);
        e = rq.xf32 ? launch_kernel(k_moe_sort_rows<true>, grid, block, 0, st, nullptr, nullptr, s, rq)
                    : launch_kernel(k_moe_sort_rows<false>, grid, block, 0, st, nullptr, nullptr, s, rq);
    } else {
        e = launch_moe_sort(a->ids, n, E, offsets, order, pos, (int32_t*)(ws + L.sort), st);
        if (e != hipSuccess) return e;
        if (per) {
            rq.nrows = offsets + E;
            rq.order = order;
            rq.topk = topk;
            rq.ids = a->ids;
            rq.s_stride = a->gate_up.s_stride;
        }
        e = launch_quantize_rows(rq, st);
    }
    if (e != hipSuccess) return e;
    I8Product p{q, a->K, qs, n, a->K, a->gate_up.codes, a->K, a->gate_up.scale, a->I, h, a->I};
    p.offsets = offsets;
    p.order = per ? nullptr : order;
    p.topk = topk;
    p.xrows = a->T;
    p.E = E;
    p.w_stride = 2 * a->I * a->K;
    p.s_down = a->down.s;
    p.s_stride = a->down.s_stride;
    p.act = a->act;
    if ((e = launch_i8_product(p, true, nullptr, st)) != hipSuccess) return e;
    I8RowsArgs rh{h, true, a->I, n, a->I, nullptr, false, hq, a->I, hs};
    rh.nrows = offsets + E;
    if ((e = launch_quantize_rows(rh, st)) != hipSuccess) return e;
    I8Product d{hq, a->I, hs, n, a->I, a->down.codes, a->I, a->down.scale, a->M, h, row_floats(a->M)};
    d.offsets = offsets;
    d.E = E;
    d.w_stride = a->M * a->I;
    if ((e = launch_i8_product(d, true, nullptr, st)) != hipSuccess) return e;
    return launch_moe_combine(h, true, n, row_floats(a->M), pos, a->w, a->T, topk, a->M, a->Y, a->yt == TTQ_F32, a->ldy, st);
}

}  // namespace ttq
