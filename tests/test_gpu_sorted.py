"""Tokens sorted by expert, their rows, and the way back with its gradient."""
import numpy as np
import pytest
import torch

import i8_ref as ref
import oracle
from gpu_util import f32_dev, host, i32_dev, say
from test_gpu_i8 import DT, enc, rounded, untouched, within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def T():
    from online_activation_aware_amd import ttq
    ttq.lib()
    return ttq


@pytest.mark.parametrize("Tn,topk,E", [(0, 2, 5), (1, 1, 1), (1, 2, 8), (7, 3, 1), (16, 2, 8), (21, 3, 64), (64, 1, 63), (100, 6, 65), (170, 6, 160),
                                       (512, 2, 1024), (1000, 32, 1023), (3000, 3, 7), (8192, 6, 160), (300001, 1, 16)])
@pytest.mark.parametrize("kind", ["even", "few", "none"])
def test_sort(T, Tn, topk, E, kind):
    say(f"moe_sort T={Tn} topk={topk} E={E} {kind}")
    rng = np.random.default_rng(Tn + E)
    ids = rng.integers(0, E, (Tn, topk)).astype(np.int32)
    if kind == "few":                                   # most slots of one expert or of none
        ids = np.where(rng.random(ids.shape) < 0.6, E // 2, ids)
        ids = np.where(rng.random(ids.shape) < 0.3, rng.choice([-1, E, E + 1, 2 ** 31 - 1, -2 ** 31], ids.shape), ids).astype(np.int32)
    if kind == "none":
        ids[:] = -1
    ws = torch.full((T.ttq_moe_sort_workspace_bytes(Tn, topk, E),), 0xEE, dtype=torch.uint8, device="cuda")
    offsets, order, pos = T.ttq_moe_sort(i32_dev(ids), E, ws=ws)
    want = ref.sort(ids, E)
    for got, w in zip((offsets, order, pos), want):
        np.testing.assert_array_equal(host(got), w)


def slots(rng, Tn, topk, rows):
    """pos of Tn x topk slots over `rows` rows, a third of them without one."""
    n = Tn * topk
    pos = np.full(n, -1, np.int64)
    have = rng.permutation(n)[: min(rows, 2 * n // 3 + 1)]
    pos[have] = rng.permutation(rows)[: have.size]
    pos[pos < 0] = rng.choice([-1, rows, rows + 7, -2 ** 31, 2 ** 31 - 1], (pos < 0).sum())
    return pos.astype(np.int32).reshape(Tn, topk)


MOVES = [(1, 1, 1, 1), (2, 3, 7, 6), (5, 2, 768, 9), (33, 4, 130, 100), (70, 1, 1027, 64), (9, 32, 264, 288), (300, 2, 4096, 600)]


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("Tn,topk,K,rows", MOVES)
def test_gather(T, dt, Tn, topk, K, rows):
    say(f"moe_gather {dt} T={Tn} topk={topk} K={K} rows={rows}")
    rng = np.random.default_rng(K + rows)
    X, x = enc(rng.standard_normal((Tn, K)), dt)
    pos = slots(rng, Tn, topk, rows)
    pad = 8 + -K % 8
    _, Xs = within(X, pad, float("nan"))
    big, R = within(torch.full((rows, K), 5.0, dtype=DT[dt], device="cuda"), pad, -3.0)
    T.ttq_moe_gather(Xs, i32_dev(pos), R=R)
    want = torch.full((rows, K), 5.0, dtype=DT[dt], device="cuda")
    for t in range(Tn):
        for j in range(topk):
            if 0 <= pos[t, j] < rows:
                want[pos[t, j]] = X[t]
    assert torch.equal(R, want) and untouched(big, R, -3.0)


@pytest.mark.parametrize("rt,yt", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("Tn,topk,M,rows", MOVES)
@pytest.mark.parametrize("weighted", [True, False])
def test_combine(T, rt, yt, Tn, topk, M, rows, weighted):
    say(f"moe_combine {rt} {yt} T={Tn} topk={topk} M={M} rows={rows} weighted={weighted}")
    rng = np.random.default_rng(M + rows)
    R, r = enc(rng.standard_normal((rows, M)), rt)
    pos = slots(rng, Tn, topk, rows)
    have = (pos >= 0) & (pos < rows)
    w = rng.standard_normal((Tn, topk)).astype(np.float32)
    wv = np.where(have, w if weighted else 1, 0).astype(np.float64)
    _, Rs = within(R, 8 + -M % 8, float("nan"))
    terms = wv[:, :, None] * r[np.where(have, pos, 0)]
    want, size = terms.sum(1), np.abs(terms).sum(1)
    bound = topk * 2.0 ** -24 * size                     # a rounding a term
    if yt == "bf16":
        bound = bound + 2.0 ** -8 * (np.abs(want) + bound)
    for pad in (0, 1, 4):
        big, Y = within(torch.empty((Tn, M), dtype=DT[yt], device="cuda"), pad, -3.0)
        wt = f32_dev(np.where(have, w, np.nan)) if weighted else None   # weights without a row are not read
        T.ttq_moe_combine(Rs, i32_dev(pos), wt, Y=Y)
        got = host(Y)
        got = oracle.decode(got, "bf16") if yt == "bf16" else got.astype(np.float64)
        assert np.all(np.abs(got - want) <= bound + 1e-40)
        assert untouched(big, Y, -3.0)


@pytest.mark.parametrize("rt,yt", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("Tn,topk,M,rows", MOVES + [(3, 2, 20001, 6)])
@pytest.mark.parametrize("weighted", [True, False])
def test_combine_grad(T, rt, yt, Tn, topk, M, rows, weighted):
    say(f"moe_combine_grad {rt} {yt} T={Tn} topk={topk} M={M} rows={rows} weighted={weighted}")
    rng = np.random.default_rng(M + rows)
    R, r = enc(rng.standard_normal((rows, M)), rt)
    dY, g = enc(rng.standard_normal((Tn, M)), yt)
    pos = slots(rng, Tn, topk, rows)
    have = (pos >= 0) & (pos < rows)
    w = rng.standard_normal((Tn, topk)).astype(np.float32)
    pad = 8 + -M % 8
    _, Rs = within(R, pad, float("nan"))
    _, dYs = within(dY, pad, float("nan"))
    big, dR = within(torch.full((rows, M), 5.0, dtype=DT[rt], device="cuda"), pad, -3.0)
    wt = f32_dev(np.where(have, w, np.nan)) if weighted else None
    dw = torch.full((Tn, topk), 9.0, device="cuda")
    T.ttq_moe_combine_grad(dYs, Rs, i32_dev(pos), wt, dR=dR, dw=dw)
    # dR: one fp32 product, rounded to its type: exact.
    want = np.full((rows, M), 5.0, np.float32)
    for t, j in zip(*np.nonzero(have)):
        want[pos[t, j]] = g[t].astype(np.float32) * (w[t, j] if weighted else np.float32(1))
    np.testing.assert_array_equal(host(dR), rounded(want, rt))
    assert untouched(big, dR, -3.0)
    # dw: no sum is longer than a sixty-fourth of the row and the sums of 64 lanes.
    terms = np.where(have[:, :, None], g[:, None] * r[np.where(have, pos, 0)], 0)
    bound = (M / 64 + 16) * 2.0 ** -24 * np.abs(terms).sum(2)
    got = host(dw).astype(np.float64)
    assert np.all(np.abs(got - terms.sum(2)) <= bound)
    assert np.all(got[~have] == 0)


def test_no_rows_at_all(T):
    say("rows 0")
    pos = i32_dev(np.zeros((3, 2)))
    none = torch.empty((0, 40), device="cuda")
    assert torch.equal(T.ttq_moe_combine(none, pos), torch.zeros((3, 40), device="cuda"))
    dY = torch.ones((3, 40), device="cuda")
    dR, dw = T.ttq_moe_combine_grad(dY, none, pos)
    assert dR.shape == (0, 40) and torch.count_nonzero(dw) == 0
    assert T.ttq_moe_gather(dY, pos, R=none) is none
    few = i32_dev(np.zeros((0, 2)))
    assert T.ttq_moe_combine(dY, few).shape == (0, 40) and T.ttq_moe_gather(dY[:0], few).shape == (0, 40)


def test_grad_parts(T):
    """dR or dw alone, through the C call."""
    say("combine_grad parts")
    rng = np.random.default_rng(5)
    dY, R = f32_dev(rng.standard_normal((6, 64))), f32_dev(rng.standard_normal((12, 64)))
    pos = i32_dev(rng.permutation(12).reshape(6, 2))
    dR, dw = T.ttq_moe_combine_grad(dY, R, pos)
    st = torch.cuda.current_stream().cuda_stream
    a, b = torch.zeros_like(dR), torch.zeros_like(dw)
    L = T.lib()
    head = (dY.data_ptr(), 0, 6, 64, 64)
    assert L.ttq_moe_combine_grad(*head, None, 0, 12, 64, pos.data_ptr(), None, 2, a.data_ptr(), 64, None, st) == 0
    assert L.ttq_moe_combine_grad(*head, R.data_ptr(), 0, 12, 64, pos.data_ptr(), None, 2, None, 0, b.data_ptr(), st) == 0
    assert torch.equal(a, dR) and torch.equal(b, dw)


def test_gradients_against_differences(T):
    """f = sum c Y of gather, experts that scale, combine: its gradients by
    both backward calls against central differences of the forward calls.  f
    is linear in X and in w, so the difference quotient is exact but for
    roundings: 2^-24 of |f| a call over a step of 1 (each term's size)."""
    say("gradients against differences")
    rng = np.random.default_rng(2)
    Tn, topk, E, K = 5, 2, 3, 24
    ids = rng.integers(0, E, (Tn, topk)).astype(np.int32)
    ids[1, 0] = -1
    _, order, pos = T.ttq_moe_sort(i32_dev(ids), E)
    x, w, c = rng.standard_normal((Tn, K)), rng.random((Tn, topk)), rng.standard_normal((Tn, K))
    x, w, c = (a.astype(np.float32) for a in (x, w, c))
    slot = host(order)
    factor = np.where(slot[:, None] >= 0, 1 + ids.reshape(-1)[slot][:, None], 0).astype(np.float32)

    def rows(x):
        R = torch.zeros((Tn * topk, K), device="cuda")
        return T.ttq_moe_gather(f32_dev(x), pos, R=R) * f32_dev(factor)

    def f(x, w):
        return float((host(T.ttq_moe_combine(rows(x), pos, f32_dev(w))).astype(np.float64) * c).sum())
    R = rows(x)
    dR, dw = T.ttq_moe_combine_grad(f32_dev(c), R, pos, f32_dev(w), dR=torch.zeros_like(R))
    dX = T.ttq_moe_combine(dR * f32_dev(factor), pos)
    size = 8 * 2.0 ** -24 * float((np.abs(host(T.ttq_moe_combine(rows(np.abs(x) + 1), pos, f32_dev(np.abs(w) + 1)))) * np.abs(c)).sum())
    for t in range(Tn):
        for k in range(0, K, 5):
            d = np.zeros_like(x)
            d[t, k] = 1
            assert abs((f(x + d, w) - f(x - d, w)) / 2 - float(dX[t, k])) <= size
        for j in range(topk):
            d = np.zeros_like(w)
            d[t, j] = 1
            assert abs((f(x, w + d) - f(x, w - d)) / 2 - float(dw[t, j])) <= size


def test_a_layer_of_the_sorted_rows(T):
    """Router, sort, gather, each expert's 8-bit product, combine: the run of
    calls gives what ttq_moe_i8's parts give, and a captured graph of it the
    same each time."""
    say("sorted layer, captured")
    rng = np.random.default_rng(9)
    Tn, E, topk, K, M = 90, 5, 2, 128, 96
    logits = f32_dev(rng.standard_normal((Tn, E)))
    X, x = enc(rng.standard_normal((Tn, K)), "bf16")
    wq = rng.integers(-127, 128, (E, M, K)).astype(np.int8)
    wsc = (rng.random((E, M)) * 0.01).astype(np.float32)
    W, ws = torch.from_numpy(wq).cuda(), f32_dev(wsc)
    ids, wt = T.ttq_moe_route(logits, topk, renormalize=True)
    at = np.concatenate(([0], np.cumsum(np.bincount(host(ids).reshape(-1), minlength=E))))
    R = torch.zeros((Tn * topk, K), dtype=torch.bfloat16, device="cuda")
    out = torch.zeros((Tn * topk, M), device="cuda")
    Y = torch.zeros((Tn, M), device="cuda")

    def run():
        T.ttq_moe_route(logits, topk, renormalize=True, ids=ids, w=wt)
        offsets, order, pos = T.ttq_moe_sort(ids, E)
        T.ttq_moe_gather(X, pos, R=R)
        for e in range(E):
            if at[e] < at[e + 1]:
                T.ttq_qgemm_i8(R[at[e]:at[e + 1]], None, W[e], ws[e], Y=out[at[e]:at[e + 1]])
        T.ttq_moe_combine(out, pos, wt, Y=Y)
    run()
    eager = Y.clone()
    q, sc = ref.quantize(x)
    want = np.zeros((Tn, M))
    size = np.zeros((Tn, M))
    for t in range(Tn):
        for j in range(topk):
            e = host(ids)[t, j]
            v = ref.product(q[t:t + 1], sc[t:t + 1], wq[e], wsc[e])[0].astype(np.float64) * host(wt)[t, j]
            want[t] += v
            size[t] += np.abs(v)
    assert np.all(np.abs(host(eager) - want) <= topk * 2.0 ** -24 * size)
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        run()
    for i in range(4):
        Y.fill_(float("nan"))
        R.fill_(float("nan"))
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(Y, eager), i
        (X.float() + 1).sum().item()                      # the program's own work between replays
