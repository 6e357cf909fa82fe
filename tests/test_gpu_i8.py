"""Linear layers in 8-bit integers: rows, products and the expert layer.
Rows and products are exact: codes, scales and results equal the reference's
bit for bit."""
import numpy as np
import pytest
import torch

import i8_ref as ref
import oracle
from gpu_util import f32_dev, host, i32_dev, say, to_dev
from online_activation_aware_amd import synth

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def T():
    from online_activation_aware_amd import ttq
    ttq.lib()
    return ttq


def enc(a, dt):
    """(device tensor, fp64 values) of an array rounded to dt."""
    e = synth.encode(np.asarray(a, np.float64), dt)
    return to_dev(e, dt), oracle.decode(e, dt)


def i8_dev(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int8)).to("cuda")


def within(t, pad, fill):
    """A matrix of t's shape within a larger one filled with `fill`: rows of
    `pad` more values, a row before and one behind."""
    big = torch.full((t.shape[0] + 2, t.shape[1] + pad), fill, dtype=t.dtype, device="cuda")
    part = big[1:-1, :t.shape[1]]
    part.copy_(t)
    return big, part


def untouched(big, part, fill):
    """The cells around `part` still hold `fill`."""
    rest = big.clone()
    rest[1:-1, :part.shape[1]] = fill
    return torch.equal(rest, torch.full_like(rest, fill))


def rounded(y, dt):
    """fp32 results as Y holds them."""
    return np.asarray(y, np.float32) if dt == "f32" else synth.encode(np.asarray(y, np.float64), "bf16")


def same(t, want):
    """Equal numbers, NaN equal to NaN."""
    got = host(t)
    if got.dtype == np.uint16:
        n = (got & 0x7FFF) > 0x7F80
        m = (want & 0x7FFF) > 0x7F80
    else:
        n, m = np.isnan(got), np.isnan(want)
    np.testing.assert_array_equal(n, m)
    np.testing.assert_array_equal(np.where(n, 0, got), np.where(m, 0, want))


# ------------------------------------------------------------------ rows

@pytest.mark.parametrize("xt", ["f32", "bf16"])
@pytest.mark.parametrize("R,K", [(1, 16), (3, 48), (5, 768), (2, 1040), (4, 4096), (700, 64), (3, 14336), (2, 16400), (1, 40016)])
@pytest.mark.parametrize("mode", ["plain", "times", "by"])
def test_quantize_rows(T, xt, R, K, mode):
    say(f"quantize_rows {xt} R={R} K={K} {mode}")
    rng = np.random.default_rng(R + K)
    X, x = enc(rng.standard_normal((R, K)) * np.where(rng.random(K) < 0.02, 30, 1), xt)
    s = None if mode == "plain" else np.exp(rng.standard_normal(K) * 0.7).astype(np.float32)
    big, part = within(torch.empty((R, K), dtype=torch.int8, device="cuda"), 32, 99)
    _, Xs = within(X, 8, float("nan"))
    codes, scale = T.ttq_quantize_rows(Xs, None if s is None else f32_dev(s), divide=mode == "by", codes=part)
    q, sc = ref.quantize(x, s, mode == "by")
    same(scale, sc)
    np.testing.assert_array_equal(host(codes), q)
    assert untouched(big, part, 99)


def test_rows_on_and_next_to_borders(T):
    """Quotients of a half, and the fp32 numbers next to them."""
    say("quantize_rows borders")
    rows = []
    for top in (127.0, 254.0, 126.99999, 3.0, 1e-3, 12345.678, 2.0 ** -90, 2.0 ** 100):
        scale = np.float32(np.float32(top) / np.float32(127))
        mid = (np.arange(-127, 127) + 0.5) * np.float64(scale)
        near = mid.astype(np.float32)
        up, down = np.nextafter(near, np.float32(np.inf)), np.nextafter(near, np.float32(-np.inf))
        row = np.concatenate(([top], near, up, down, [0, -0.0]))
        rows.append(np.concatenate((row, np.zeros(768 - row.size))))
    x = np.array(rows, np.float32)
    codes, scale = T.ttq_quantize_rows(f32_dev(x))
    q, sc = ref.quantize(x)
    same(scale, sc)
    np.testing.assert_array_equal(host(codes), q)


def test_rows_without_a_range(T):
    """Zeros, subnormal rows, the largest numbers; infinities and NaN spoil
    their own row only."""
    say("quantize_rows extremes")
    rng = np.random.default_rng(3)
    x = rng.standard_normal((14, 80)).astype(np.float32)
    tiny = np.float32(2.0 ** -149)
    x[0] = 0
    x[1] = -0.0
    x[2] = tiny * rng.integers(-50, 51, 80)            # the scale rounds to zero: 1
    x[3] = tiny * rng.integers(-190, 191, 80)          # ... to one step: codes clamp
    x[3, 5] = tiny * 190
    x[4] = tiny * rng.integers(-90000, 90001, 80)
    x[5] *= np.float32(2.0 ** -126)
    x[6] = np.finfo(np.float32).max
    x[7] *= np.float32(1e38)
    x[8, 3] = np.inf
    x[9, 79] = -np.inf
    x[10, 0] = np.nan
    x[11, 40] = np.finfo(np.float32).min
    x[12] = 1
    s = np.ones(80, np.float32)
    s[7] = 2.0 ** -130
    for sv, divide in ((None, False), (s, True), (s, False)):
        codes, scale = T.ttq_quantize_rows(f32_dev(x), None if sv is None else f32_dev(sv), divide=divide)
        q, sc = ref.quantize(x, sv, divide)
        same(scale, sc)
        np.testing.assert_array_equal(host(codes), q)


# ------------------------------------------------------------------ products

SHAPES = [(1, 16, 1), (1, 64, 17), (1, 4096, 300), (2, 48, 16), (3, 80, 33), (4, 1040, 65), (5, 112, 3), (8, 14336, 40), (15, 768, 130),
          (16, 2064, 257), (17, 128, 100), (31, 176, 64), (33, 4112, 48), (48, 256, 513), (64, 1088, 200), (65, 320, 129), (100, 96, 258),
          (128, 768, 768), (130, 2048, 70), (200, 144, 1411), (257, 640, 256), (300, 1056, 515), (513, 400, 260), (1030, 272, 130), (8, 131072, 5)]


@pytest.mark.parametrize("Tn,K,M", SHAPES)
@pytest.mark.parametrize("yt", ["f32", "bf16"])
def test_gemm(T, Tn, K, M, yt):
    say(f"gemm_i8 T={Tn} K={K} M={M} {yt}")
    rng = np.random.default_rng(Tn + K + M)
    xq, wq = rng.integers(-127, 128, (Tn, K)), rng.integers(-127, 128, (M, K))
    xq[0] = 127                                          # the largest sums
    wq[0] = 127
    wq[-1] = -127
    xs, ws = rng.random(Tn).astype(np.float32), rng.random(M).astype(np.float32)
    want = rounded(ref.product(xq, xs, wq, ws), yt)
    _, X = within(i8_dev(xq), 16, 77)
    _, W = within(i8_dev(wq), 48, 88)
    for pad in (0, 4, 5):
        big, Y = within(torch.empty((Tn, M), dtype=DT[yt], device="cuda"), pad, -3.0)
        T.ttq_gemm_i8(X, f32_dev(xs), W, f32_dev(ws), Y=Y)
        same(Y, want)
        assert untouched(big, Y, -3.0)


@pytest.mark.parametrize("Tn,K,M", [(1, 4096, 300), (2, 768, 768), (4, 1040, 65), (7, 14336, 130), (16, 4096, 257), (40, 2064, 96),
                                    (128, 768, 768), (300, 1056, 515), (1, 40016, 24)])
@pytest.mark.parametrize("xt,yt", [("bf16", "bf16"), ("f32", "f32"), ("bf16", "f32")])
@pytest.mark.parametrize("scaled", [True, False])
def test_qgemm(T, Tn, K, M, xt, yt, scaled):
    say(f"qgemm_i8 T={Tn} K={K} M={M} {xt} {yt} scaled={scaled}")
    rng = np.random.default_rng(Tn + K + M)
    X, x = enc(rng.standard_normal((Tn, K)) * np.where(rng.random(K) < 0.02, 30, 1), xt)
    s = np.exp(rng.standard_normal(K) * 0.5).astype(np.float32) if scaled else None
    w = rng.standard_normal((M, K)).astype(np.float32)
    W, ws = T.ttq_quantize_rows(f32_dev(w), None if s is None else f32_dev(s))
    wq, wsc = ref.quantize(w, s)
    np.testing.assert_array_equal(host(W), wq)
    want = rounded(ref.product(*ref.quantize(x, s, True), wq, wsc), yt)
    Y = T.ttq_qgemm_i8(X, None if s is None else f32_dev(s), W, ws, y_dtype=DT[yt])
    same(Y, want)


@pytest.mark.parametrize("K,M", [(16, 1), (48, 33), (80, 17), (144, 6161), (320, 12300), (1040, 4097), (16384, 40), (16400, 40)])
@pytest.mark.parametrize("xt,yt", [("bf16", "bf16"), ("f32", "f32")])
def test_qgemm_one_token(T, K, M, xt, yt):
    """One launch: fewer channels than its waves take at once, several turns of
    one, two and four blocks; more channels than it holds."""
    say(f"qgemm_i8 one token K={K} M={M} {xt} {yt}")
    rng = np.random.default_rng(K + M)
    X, x = enc(rng.standard_normal((1, K)), xt)
    s = np.exp(rng.standard_normal(K) * 0.5).astype(np.float32)
    wq = rng.integers(-127, 128, (M, K)).astype(np.int8)
    ws = rng.random(M).astype(np.float32)
    big, Y = within(torch.empty((1, M), dtype=DT[yt], device="cuda"), 3, -3.0)
    for sv in (s, None):
        T.ttq_qgemm_i8(X, None if sv is None else f32_dev(sv), i8_dev(wq), f32_dev(ws), Y=Y)
        same(Y, rounded(ref.product(*ref.quantize(x, sv, True), wq, ws), yt))
        assert untouched(big, Y, -3.0)


@pytest.mark.parametrize("Tn", [1, 3, 20, 200])
def test_qgemm_rows_that_are_not_finite(T, Tn):
    say(f"qgemm_i8 not finite T={Tn}")
    rng = np.random.default_rng(Tn)
    x = rng.standard_normal((Tn, 320)).astype(np.float32)
    x[Tn // 2, 300] = np.nan
    if Tn > 3:
        x[5, 0], x[6, 319] = np.inf, -np.inf
        x[7] = 0
    w = rng.standard_normal((70, 320)).astype(np.float32)
    wq, ws = ref.quantize(w)
    want = ref.product(*ref.quantize(x), wq, ws)
    same(T.ttq_qgemm_i8(f32_dev(x), None, i8_dev(wq), f32_dev(ws)), want)


def test_products_of_no_rows(T):
    say("gemm_i8 empty")
    w = i8_dev(np.ones((5, 32)))
    one = torch.ones(5, device="cuda")
    none = torch.empty((0, 32), dtype=torch.int8, device="cuda")
    assert T.ttq_gemm_i8(none, one[:0], w, one).shape == (0, 5)
    assert T.ttq_gemm_i8(w, one, none, one[:0]).shape == (5, 0)
    assert T.ttq_qgemm_i8(torch.empty((0, 32), device="cuda"), None, w, one).shape == (0, 5)
    q, s = T.ttq_quantize_rows(torch.empty((0, 32), device="cuda"))
    assert q.shape == (0, 32) and s.shape == (0,)


# ------------------------------------------------------------------ experts

def moe_inputs(seed, Tn, E, topk, K, I, M, xt, per_in, per_down, drop):
    rng = np.random.default_rng(seed)
    X, x = enc(rng.standard_normal((Tn, K)) * np.where(rng.random(K) < 0.05, 20, 1), xt)
    ids = rng.integers(0, E, (Tn, topk)).astype(np.int32)
    if drop:
        ids[rng.random(ids.shape) < 0.3] = -1
        ids[0] = E                                       # a token without any expert
    w = rng.random((Tn, topk)).astype(np.float32)
    d = dict(X=X, x=x, ids=ids, w=w)
    for key, rows, cols, per in (("gate_up", 2 * I, K, per_in), ("down", M, I, per_down)):
        q = rng.integers(-127, 128, (E, rows, cols)).astype(np.int8)
        sc = (rng.random((E, rows)) * 0.02 / np.sqrt(cols) + 1e-4).astype(np.float32)
        s = np.exp(rng.standard_normal((E, cols) if per else cols) * 0.5).astype(np.float32)
        d[key] = dict(s=f32_dev(s), codes=i8_dev(q), scale=f32_dev(sc))
        d[key + "_ref"] = (q, sc, s)
    return d


def moe_ref(d, act):
    (gu, gs, s_in), (dn, ds, s_down) = d["gate_up_ref"], d["down_ref"]
    ids = d["ids"]
    per = s_in.ndim == 2
    if per:
        Tn, k = ids.shape
        e = np.clip(ids, 0, s_in.shape[0] - 1)
        q, sc = ref.quantize(np.repeat(d["x"], k, 0), s_in[e.reshape(-1)], True)
        q, sc = q.reshape(Tn, k, -1), sc.reshape(Tn, k)
    else:
        q, sc = ref.quantize(d["x"], s_in, True)
    return ref.moe(q, sc, per, ids, d["w"].astype(np.float64), gu, gs, s_down, dn, ds, act)


def near(Y, want, bound, yt):
    got = host(Y)
    got = oracle.decode(got, "bf16") if yt == "bf16" else got.astype(np.float64)
    if yt == "bf16":
        bound = bound + 2.0 ** -8 * (np.abs(want) + bound)   # half a step of the result
    off = np.abs(got - want) - bound - 1e-37
    assert np.all(off <= 0), float(off.max())


MOE = [  # T, E, topk, K, I, M, xt, yt, act, per_in, per_down, drop
    (1, 1, 1, 16, 16, 1, "f32", "f32", "silu", False, False, False),
    (1, 8, 2, 256, 384, 256, "bf16", "bf16", "silu", False, True, False),
    (2, 4, 4, 48, 80, 33, "f32", "f32", "gelu", True, False, False),
    (5, 4, 2, 768, 2048, 96, "f32", "f32", "gelu", False, True, True),
    (16, 64, 6, 160, 112, 65, "bf16", "f32", "silu", False, True, False),
    (33, 3, 2, 320, 272, 130, "bf16", "bf16", "silu", True, True, True),
    (64, 2, 2, 528, 144, 100, "bf16", "f32", "gelu", False, False, False),
    (130, 9, 4, 64, 96, 70, "f32", "bf16", "silu", True, True, True),
    (300, 5, 3, 144, 176, 258, "bf16", "f32", "silu", False, True, True),
    (700, 3, 2, 96, 80, 129, "bf16", "bf16", "silu", False, True, False),
    (90, 200, 8, 32, 48, 17, "f32", "f32", "silu", False, True, True),
    (40, 1024, 32, 32, 16, 8, "bf16", "f32", "silu", False, True, False),
]


@pytest.mark.parametrize("case", MOE, ids=lambda c: "-".join(map(str, c)))
def test_moe(T, case):
    Tn, E, topk, K, I, M, xt, yt, act, per_in, per_down, drop = case
    say(f"moe_i8 {case}")
    d = moe_inputs(sum(case[:6]), Tn, E, topk, K, I, M, xt, per_in, per_down, drop)
    n = T.ttq_moe_i8_workspace_bytes(Tn, topk, K, I, M, E)
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")     # NaN wherever it is read before it is written
    big, Y = within(torch.empty((Tn, M), dtype=DT[yt], device="cuda"), 3, -3.0)
    T.ttq_moe_i8(d["X"], i32_dev(d["ids"]), f32_dev(d["w"]), d["gate_up"], d["down"], act=act, Y=Y, ws=ws)
    want, bound = moe_ref(d, act)
    near(Y, want, bound, yt)
    assert untouched(big, Y, -3.0)


def test_moe_all_tokens_to_one_expert_and_none(T):
    say("moe_i8 one expert, none")
    d = moe_inputs(7, 150, 6, 2, 128, 96, 64, "bf16", False, True, False)
    for ids in (np.full((150, 2), 4, np.int32), np.full((150, 2), -1, np.int32), np.full((150, 2), 6, np.int32)):
        d["ids"] = ids
        Y = T.ttq_moe_i8(d["X"], i32_dev(ids), f32_dev(np.where(ids == 4, d["w"], np.nan)), d["gate_up"], d["down"])
        if ids[0, 0] != 4:
            assert torch.count_nonzero(Y) == 0
        else:
            near(Y, *moe_ref(d, "silu"), "f32")


@pytest.mark.parametrize("Tn", [3, 60, 400])
def test_moe_tokens_that_are_not_finite(T, Tn):
    say(f"moe_i8 not finite T={Tn}")
    d = moe_inputs(Tn, Tn, 4, 2, 128, 96, 64, "f32", False, True, False)
    args = (i32_dev(d["ids"]), f32_dev(d["w"]), d["gate_up"], d["down"])
    clean = T.ttq_moe_i8(d["X"], *args)
    X = d["X"].clone()
    X[1, 5] = float("nan")
    X[2, 100] = float("inf")
    X[0] = 3e38                                          # h overflows
    Y = T.ttq_moe_i8(X, *args)
    assert torch.isnan(Y[1]).all() and torch.isnan(Y[2]).all() and not torch.isfinite(Y[0]).any()
    assert torch.equal(Y[3:], clean[3:])


def test_moe_token_alone_and_in_company(T):
    """A token's results do not depend on the others of the call."""
    say("moe_i8 alone")
    d = moe_inputs(11, 520, 4, 2, 256, 192, 130, "bf16", False, True, False)
    ids, w = i32_dev(d["ids"]), f32_dev(d["w"])
    every = T.ttq_moe_i8(d["X"], ids, w, d["gate_up"], d["down"])
    for n in (1, 2, 9, 40, 100, 260):
        part = T.ttq_moe_i8(d["X"][:n], ids[:n].contiguous(), w[:n].contiguous(), d["gate_up"], d["down"])
        assert torch.equal(part, every[:n]), n
