"""Projections whose weights each token chooses: the expert router, the
mixture-of-experts layer on quantized experts, adapters of many requests, and
a shared projection with adapters, element by element against fp64."""
import math

import numpy as np
import pytest
import torch

import oracle
import routed_ref as ref
from gpu_util import bf16_bits_to_f64, f32_dev, host, i32_dev, say, to_dev
from online_activation_aware_amd import synth

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def T():
    from online_activation_aware_amd import ttq
    ttq.lib()
    return ttq


def num(t):
    """A device tensor's values in fp64."""
    h = host(t)
    return bf16_bits_to_f64(h) if t.dtype == torch.bfloat16 else h.astype(np.float64)


def enc(a, dt):
    """(device tensor, fp64 values) of an array rounded to dt."""
    e = synth.encode(np.asarray(a, np.float64), dt)
    return to_dev(e, dt), oracle.decode(e, dt)


# ------------------------------------------------------------------ router

@pytest.mark.parametrize("lt", ["f32", "bf16"])
@pytest.mark.parametrize("Tn,E,topk", [(1, 1, 1), (3, 8, 2), (5, 8, 8), (70, 64, 6), (9, 65, 4), (33, 160, 6), (4, 256, 32),
                                       (2, 511, 3), (2, 1024, 32)])
@pytest.mark.parametrize("score,renorm", [("softmax", False), ("softmax", True), ("sigmoid", False), ("sigmoid", True)])
def test_route(T, lt, Tn, E, topk, score, renorm):
    say(f"route {lt} T={Tn} E={E} topk={topk} {score} renorm={renorm}")
    rng = np.random.default_rng(E + topk)
    L, x = enc(rng.standard_normal((Tn, E)) * 3, lt)
    ids, w = T.ttq_moe_route(L, topk, score=score, renormalize=renorm)
    ri, rw, rb = ref.route(x, topk, score, renorm)
    np.testing.assert_array_equal(host(ids), ri)
    assert np.all(np.abs(num(w) - rw) <= rb * rw + 1e-37)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_masks_ties_and_infinities(T, score):
    say(f"route masks {score}")
    inf, nan, low = np.inf, np.nan, -3.3895313892515355e38   # the lowest bf16
    rows = [[-inf] * 6, [nan] * 6, [nan, -inf, 2, -inf, nan, 1], [1, 1, 1, 1, 1, 1], [low] * 6, [low, 0, low, -inf, low, low],
            [inf, 1, inf, 2, -inf, 3], [-0.0, 0.0, -0.0, -1, -2, nan], [5, -inf, -inf, -inf, -inf, -inf], [-1e38, 1e38, 0, 3, 3, 2]]
    x = np.array(rows, np.float64)
    big = torch.full((len(rows), 11), 7.0, device="cuda")        # rows of a wider matrix
    big[:, :6] = f32_dev(x)
    for L, v in ((big[:, :6], x.astype(np.float32).astype(np.float64)), enc(x, "bf16")):
        for renorm in (False, True):
            ids, w = T.ttq_moe_route(L, 4, score=score, renormalize=renorm)
            ri, rw, rb = ref.route(v, 4, score, renorm)
            np.testing.assert_array_equal(host(ids), ri)
            assert np.all(np.abs(num(w) - rw) <= rb * rw + 1e-37)


# ------------------------------------------------------------------ experts

def moe_inputs(seed, Tn, E, topk, K, I, M, bits, group, xt, per_in=False, per_down=True):
    rng = np.random.default_rng(seed)
    X, x = enc(rng.standard_normal((Tn, K)) * np.where(rng.random(K) < 0.05, 20, 1), xt)
    w = rng.random((Tn, topk)).astype(np.float32)
    ids = rng.integers(0, E, (Tn, topk)).astype(np.int32)
    out = dict(X=X, x=x, w=w, ids=ids)
    for key, rows, cols, per in (("gate_up", 2 * I, K, per_in), ("down", M, I, per_down)):
        codes, step, zero, n = ref.quantized(rng, E, rows, cols, bits, group)
        s = np.exp(rng.standard_normal((E, cols) if per else cols) * 0.5).astype(np.float32)
        out[key] = dict(s=f32_dev(s), codes=i32_dev(codes), scale_f16=torch.from_numpy(step).cuda(),
                        zero_f16=torch.from_numpy(zero).cuda())
        out[key + "_ref"] = (n, s.astype(np.float64))
    return out


def moe_ref(d, bits, act, xt, group):
    (gu, s_in), (dn, s_down) = d["gate_up_ref"], d["down_ref"]
    return ref.moe(d["x"], d["ids"], d["w"].astype(np.float64), gu, s_in, dn, s_down, bits, act,
                   2.0 ** -16 if xt == "bf16" else 2.0 ** -23, group)


MOE = [  # T, E, topk, K, I, M, bits, group, xt, yt, act
    (1, 8, 2, 256, 384, 256, 4, 32, "bf16", "bf16", "silu"),
    (1, 1, 1, 32, 32, 1, 4, 32, "bf16", "f32", "silu"),
    (1, 4, 3, 544, 1056, 65, 4, 32, "bf16", "f32", "gelu"),
    (1, 6, 6, 1024, 512, 300, 4, 64, "f32", "f32", "silu"),
    (2, 3, 4, 640, 384, 129, 4, 128, "bf16", "f32", "silu"),
    (2, 40, 8, 2048, 64, 64, 4, 32, "f32", "bf16", "gelu"),
    (3, 4, 2, 96, 160, 33, 4, 32, "bf16", "f32", "gelu"),
    (7, 64, 6, 160, 96, 80, 4, 32, "bf16", "f32", "silu"),
    (16, 5, 3, 512, 640, 513, 4, 64, "bf16", "f32", "silu"),
    (17, 2, 1, 1152, 256, 64, 4, 128, "bf16", "f32", "silu"),
    (40, 3, 2, 640, 1056, 96, 4, 32, "bf16", "bf16", "gelu"),
    (130, 9, 4, 256, 288, 130, 4, 32, "bf16", "f32", "silu"),
    (300, 2, 2, 128, 128, 48, 4, 64, "bf16", "f32", "silu"),
    (5, 4, 2, 768, 512, 96, 3, 16, "f32", "f32", "gelu"),
    (2, 3, 2, 2080, 4128, 40, 4, 32, "bf16", "f32", "silu"),
    (2, 3, 2, 2080, 4128, 40, 4, 32, "f32", "f32", "silu"),
    (9, 3, 2, 256, 128, 64, 4, 16, "bf16", "f32", "silu"),
    (9, 3, 2, 256, 128, 64, 2, 32, "bf16", "f32", "silu"),
    (33, 3, 2, 256, 128, 64, 5, 128, "bf16", "f32", "gelu"),
    (6, 3, 3, 320, 192, 70, 3, 64, "bf16", "bf16", "silu"),
    (19, 6, 2, 384, 256, 100, 4, 64, "f32", "bf16", "silu"),
    # more than 16 slots an expert: 33 (one behind a tile of 32), several rounds of channels, odd numbers of groups
    (33, 1, 1, 1024, 288, 40, 4, 32, "bf16", "f32", "silu"),
    (70, 2, 2, 2048, 1408, 72, 4, 32, "bf16", "bf16", "silu"),
    (40, 2, 1, 1312, 352, 136, 4, 32, "f32", "f32", "gelu"),
    (50, 2, 2, 1024, 768, 64, 4, 128, "f32", "f32", "silu"),
    (90, 3, 2, 1536, 640, 300, 4, 64, "bf16", "f32", "silu"),
    (60, 2, 2, 1024, 512, 40, 3, 16, "f32", "f32", "gelu"),
    (60, 2, 2, 800, 544, 40, 2, 32, "bf16", "bf16", "silu"),
    (60, 2, 2, 640, 1024, 40, 5, 64, "bf16", "f32", "silu"),
]


@pytest.mark.parametrize("case", MOE, ids=lambda c: "-".join(map(str, c)))
def test_moe(T, case):
    Tn, E, topk, K, I, M, bits, group, xt, yt, act = case
    say(f"moe {case}")
    d = moe_inputs(sum(case[:8]), Tn, E, topk, K, I, M, bits, group, xt, per_in=E % 2 == 0)
    y = T.ttq_moe(d["X"], i32_dev(d["ids"]), f32_dev(d["w"]), d["gate_up"], d["down"], bits, group, act=act, y_dtype=DT[yt])
    r, b = moe_ref(d, bits, act, xt, group)
    ref.check(num(y), r, b, yt == "bf16")


@pytest.mark.parametrize("bits,group,xt", [(4, 32, "bf16"), (4, 64, "f32"), (3, 16, "bf16")])
@pytest.mark.parametrize("Tn", [1, 12, 50])
def test_moe_slots_without_an_expert_and_strides(T, bits, group, xt, Tn):
    say(f"moe slots b{bits} g{group} {xt} T={Tn}")
    E, topk, K, I, M = 4, 3, 192, 128, 70
    d = moe_inputs(Tn + bits, Tn, E, topk, K, I, M, bits, group, xt)
    ids = d["ids"]
    ids[:, 1] = -1
    if Tn > 2:
        ids[1] = 2                                 # one expert three times
        ids[2:, 0] = 3                             # a crowded expert
    ids[Tn // 2] = [E, -7, 1 << 30]                # a token without any
    w = d["w"].copy()
    w[(ids < 0) | (ids >= E)] = np.nan             # never read
    big = torch.full((Tn, K + 64), 3.0, dtype=d["X"].dtype, device="cuda")
    big[:, 32:32 + K] = d["X"]
    Y = torch.full((Tn, M + 5), -77.0, device="cuda")
    T.ttq_moe(big[:, 32:32 + K], i32_dev(ids), f32_dev(w), d["gate_up"], d["down"], bits, group, Y=Y[:, 2:2 + M])
    r, b = moe_ref(d, bits, "silu", xt, group)
    y = num(Y)
    ref.check(y[:, 2:2 + M], r, b, False)
    assert np.all(y[Tn // 2, 2:2 + M] == 0)
    assert np.all(y[:, :2] == -77) and np.all(y[:, 2 + M:] == -77)


@pytest.mark.parametrize("Tn,bits,group", [(1, 4, 32), (2, 4, 64), (12, 4, 32), (12, 4, 128), (12, 3, 32), (12, 4, 16)])
def test_moe_steps_of_other_rows_do_not_matter(T, Tn, bits, group):
    """A row whose steps and zeros are no numbers leaves the others as they are (rows end inside a chunk)."""
    say(f"moe steps b{bits} g{group} T={Tn}")
    I, M = 5 * max(group, 32), 9
    d = moe_inputs(Tn + group, Tn, 2, 2, 256, I, M, bits, group, "bf16")
    args = d["X"], i32_dev(d["ids"]), f32_dev(d["w"]), d["gate_up"]
    want = num(T.ttq_moe(*args, d["down"], bits, group))
    down = dict(d["down"], scale_f16=d["down"]["scale_f16"].clone(), zero_f16=d["down"]["zero_f16"].clone())
    down["scale_f16"][:, 4] = math.inf
    down["zero_f16"][:, 4] = math.nan
    y = num(T.ttq_moe(*args, down, bits, group))
    rows = np.arange(M) != 4
    np.testing.assert_array_equal(y[:, rows], want[:, rows])
    assert np.all(np.isnan(y[:, 4]))


@pytest.mark.parametrize("xt", ["bf16", "f32"])
@pytest.mark.parametrize("Tn", [1, 2, 12])
def test_moe_nan_stays_in_its_token(T, Tn, xt):
    say(f"moe nan {xt} T={Tn}")
    d = moe_inputs(Tn, Tn, 2, 2, 256, 160, 40, 4, 32, xt)
    args = i32_dev(d["ids"]), f32_dev(d["w"]), d["gate_up"], d["down"], 4, 32
    want = num(T.ttq_moe(d["X"], *args))
    X = d["X"].clone()
    X[0, 77] = math.nan
    y = num(T.ttq_moe(X, *args))
    assert np.all(np.isnan(y[0]))
    np.testing.assert_array_equal(y[1:], want[1:])


@pytest.mark.parametrize("Tn", [1, 2])
def test_moe_tiny_weights(T, Tn):
    """Weights of 2^-110 scale the result (the range of h's integers: their scale is 2^-129 here, off by at
    most 2^-150, a 2^-21st of it)."""
    say(f"moe tiny weights T={Tn}")
    d = moe_inputs(3, Tn, 2, 2, 256, 160, 40, 4, 32, "bf16")
    d["w"] = (d["w"] * 2.0 ** -110).astype(np.float32)
    y = T.ttq_moe(d["X"], i32_dev(d["ids"]), f32_dev(d["w"]), d["gate_up"], d["down"], 4, 32)
    r, b = moe_ref(d, 4, "silu", "bf16", 32)
    ref.check(num(y) * 2.0 ** 110, r * 2.0 ** 110, b * 2.0 ** 110, False)


def test_moe_all_slots_empty(T):
    say("moe without experts")
    d = moe_inputs(1, 6, 3, 2, 64, 64, 32, 4, 32, "bf16")
    y = T.ttq_moe(d["X"], torch.full((6, 2), -1, dtype=torch.int32, device="cuda"), f32_dev(d["w"]), d["gate_up"], d["down"],
                  4, 32)
    assert torch.count_nonzero(y) == 0


@pytest.mark.parametrize("group", [32, 128])
def test_moe_rows_do_not_depend_on_the_batch(T, group):
    """A token alone and in a batch: both within the bound of the definition,
    and repeated calls bitwise equal."""
    say(f"moe batch g{group}")
    Tn, E, topk, K, I, M = 24, 4, 2, 384, 256, 96
    d = moe_inputs(9, Tn, E, topk, K, I, M, 4, group, "bf16")
    ids, w = i32_dev(d["ids"]), f32_dev(d["w"])
    call = lambda a, b: T.ttq_moe(d["X"][a:b], ids[a:b].contiguous(), w[a:b].contiguous(), d["gate_up"], d["down"], 4, group)  # noqa: E731
    r, b = moe_ref(d, 4, "silu", "bf16", group)
    whole = call(0, Tn)
    assert torch.equal(whole, call(0, Tn))
    ref.check(num(whole), r, b, False)
    for t in (0, 7, 23):
        one = dict(d, x=d["x"][t:t + 1], ids=d["ids"][t:t + 1], w=d["w"][t:t + 1])
        r1, b1 = moe_ref(one, 4, "silu", "bf16", group)
        ref.check(num(call(t, t + 1)), r1, b1, False)
        ref.check(num(call(t, t + 1)), num(whole)[t:t + 1], b1 + b[t:t + 1], False)


# ------------------------------------------------------------------ adapters

def adapter_inputs(seed, Tn, K, M, n, rank, at, mode):
    rng = np.random.default_rng(seed)
    A, a = enc(rng.standard_normal((n, rank, K)) / np.sqrt(K), at)
    B, b = enc(rng.standard_normal((n, M, rank)), at)
    ids = rng.integers(-1, n + 1, Tn) if mode == "mixed" else np.sort(rng.integers(0, n, Tn)) if mode == "runs" else np.full(Tn, n - 1)
    ranks = rng.integers(0, rank + 1, n).astype(np.int32)
    scale = (rng.random(n) + 0.5).astype(np.float32)
    return dict(A=A, a=a, B=B, b=b, ids=ids.astype(np.int32), ranks=ranks, scale=scale, rng=rng)


ADAPTERS = [  # T, K, M, n, rank, xt, at, yt, ids
    (1, 4096, 512, 3, 16, "bf16", "bf16", "bf16", "one"),
    (1, 8, 1, 1, 1, "bf16", "bf16", "f32", "one"),
    (1, 4096, 14344, 2, 64, "bf16", "bf16", "f32", "one"),
    (1, 520, 131, 3, 13, "f32", "bf16", "f32", "one"),
    (1, 2056, 300, 3, 64, "bf16", "f32", "bf16", "one"),
    (5, 40, 33, 2, 3, "bf16", "bf16", "f32", "mixed"),
    (16, 256, 100, 7, 8, "bf16", "bf16", "f32", "mixed"),
    (33, 776, 130, 40, 32, "bf16", "bf16", "f32", "mixed"),
    (48, 1024, 515, 64, 64, "bf16", "bf16", "f32", "mixed"),
    (300, 512, 260, 4, 24, "bf16", "bf16", "f32", "runs"),
    (129, 2048, 192, 5, 64, "bf16", "bf16", "bf16", "runs"),
    (70, 256, 64, 3, 17, "bf16", "f32", "f32", "mixed"),
    (70, 264, 65, 3, 20, "f32", "bf16", "f32", "mixed"),
    (20, 768, 768, 6, 16, "f32", "f32", "f32", "mixed"),
    (200, 128, 48, 2, 40, "f32", "f32", "bf16", "runs"),
    (150, 4096, 64, 3, 64, "bf16", "bf16", "bf16", "runs"),
    (140, 3584, 136, 3, 32, "bf16", "f32", "f32", "runs"),
    (200, 2560, 72, 2, 56, "bf16", "bf16", "f32", "runs"),
    (3, 16384, 40, 2, 4, "bf16", "bf16", "f32", "mixed"),
]


@pytest.mark.parametrize("case", ADAPTERS, ids=lambda c: "-".join(map(str, c)))
@pytest.mark.parametrize("ragged", [False, True])
def test_adapters_add(T, case, ragged):
    Tn, K, M, n, rank, xt, at, yt, mode = case
    say(f"adapters {case} ragged={ragged}")
    d = adapter_inputs(sum(case[:5]), Tn, K, M, n, rank, at, mode)
    X, x = enc(d["rng"].standard_normal((Tn, K)), xt)
    C, c = enc(d["rng"].standard_normal((Tn, M)), yt)
    rk, sc = (d["ranks"], d["scale"]) if ragged else (None, None)
    if ragged:   # what lies behind a rank is not used
        for i, r in enumerate(d["ranks"]):
            d["A"][i, r:] = float("nan")
            d["B"][i, :, r:] = float("nan")
    y = T.ttq_adapters_add(X, d["A"], d["B"], i32_dev(d["ids"]), C=C, ranks=None if rk is None else i32_dev(rk),
                           scale=None if sc is None else f32_dev(sc))
    r, b = ref.adapters(x, d["a"], d["b"], d["ids"], rk, sc)
    ref.check(num(y), c + r, b + np.abs(c) * ref.U32, yt == "bf16")
    none = (d["ids"] < 0) | (d["ids"] >= n)
    assert np.array_equal(num(y)[none], c[none])
    z = T.ttq_adapters_add(X, d["A"], d["B"], i32_dev(d["ids"]), C=C, Y=C, ranks=None if rk is None else i32_dev(rk),
                           scale=None if sc is None else f32_dev(sc))
    assert z is C and torch.equal(z, y)            # in place


def test_adapters_without_a_projection_strided_and_without_adapters(T):
    say("adapters strided")
    Tn, K, M, n, rank = 37, 96, 50, 3, 12
    d = adapter_inputs(2, Tn, K, M, n, rank, "bf16", "mixed")
    X, x = enc(d["rng"].standard_normal((Tn, K)), "bf16")
    big = torch.full((Tn, K + 32), float("nan"), dtype=torch.bfloat16, device="cuda")
    big[:, 16:16 + K] = X
    Y = torch.full((Tn + 2, M + 3), -5.0, device="cuda")
    T.ttq_adapters_add(big[:, 16:16 + K], d["A"], d["B"], i32_dev(d["ids"]), Y=Y[1:-1, 1:1 + M])
    r, b = ref.adapters(x, d["a"], d["b"], d["ids"])
    y = num(Y)
    ref.check(y[1:-1, 1:1 + M], r, b, False)
    assert np.all(y[[0, -1]] == -5) and np.all(y[:, 0] == -5) and np.all(y[:, 1 + M:] == -5)
    C = torch.randn((Tn, M), device="cuda")
    e = T.ttq_adapters_add(X, d["A"][:0], d["B"][:0], i32_dev(d["ids"]), C=C)
    assert torch.equal(e, C)


# ------------------------------------------------------------------ a shared projection with adapters

SHARED = [  # T, K, M, bits, group, n, rank, xt, yt, ids
    (1, 1024, 256, 4, 32, 3, 16, "bf16", "f32", "mixed"),
    (4, 4096, 130, 4, 64, 5, 8, "bf16", "bf16", "mixed"),
    (6, 288, 70, 4, 32, 4, 5, "bf16", "bf16", "mixed"),
    (16, 2048, 192, 4, 128, 20, 64, "bf16", "bf16", "mixed"),
    (13, 512, 65, 3, 16, 4, 16, "bf16", "bf16", "mixed"),
    (16, 256, 64, 4, 32, 4, 16, "f32", "f32", "mixed"),
    (3, 160, 33, 5, 32, 2, 7, "f32", "f32", "mixed"),
    (100, 768, 96, 4, 32, 3, 16, "bf16", "bf16", "runs"),
    (260, 1024, 288, 4, 32, 4, 32, "bf16", "bf16", "runs"),
    (300, 8192, 130, 2, 32, 3, 17, "bf16", "bf16", "runs"),
    (40, 256, 64, 4, 64, 3, 16, "f32", "f32", "runs"),
]


@pytest.mark.parametrize("case", SHARED, ids=lambda c: "-".join(map(str, c)))
def test_qgemm_adapters(T, case):
    Tn, K, M, bits, group, n, rank, xt, yt, mode = case
    say(f"shared {case}")
    d = adapter_inputs(sum(case[:7]), Tn, K, M, n, rank, xt, mode)
    rng = d["rng"]
    X, x = enc(rng.standard_normal((Tn, K)), xt)
    codes, step, zero, (q, dl, z) = ref.quantized(rng, 1, M, K, bits, group)
    s = np.exp(rng.standard_normal(K) * 0.5).astype(np.float32)
    Y = torch.full((Tn, M + 3), -3.0, dtype=DT[yt], device="cuda")
    T.ttq_qgemm_adapters(X, f32_dev(s), i32_dev(codes[0]), torch.from_numpy(step[0]).cuda(), torch.from_numpy(zero[0]).cuda(),
                         M, bits, group, d["A"], d["B"], i32_dev(d["ids"]), ranks=i32_dev(d["ranks"]),
                         scale=f32_dev(d["scale"]), Y=Y[:, :M])
    # the projection kernels round the dequantized weight (or x / s) once to bf16 for bf16 X, split it in two for fp32 X
    rel = 2.0 ** -8 if xt == "bf16" else 2.0 ** -14
    w = (q[0] - z[0]) * dl[0] / s
    y = x @ w.T
    b = (np.abs(x) @ np.abs(w).T) * rel + (np.abs(x) @ (dl[0] * (q[0] + z[0] + 256) / s).T) * (2.0 ** -21 + 3 * K * ref.U32)
    r, ba = ref.adapters(x, d["a"], d["b"], d["ids"], d["ranks"], d["scale"])
    ref.check(num(Y)[:, :M], y + r, b + ba, yt == "bf16")
    assert np.all(num(Y)[:, M:] == -3)


# ------------------------------------------------------------------ together

def test_a_layer_of_routed_projections(T):
    """As a server uses them: expert weights quantized by the library with
    their shared statistics' scales, a shared projection with the requests'
    adapters, the router, the experts; eager on a stream of its own, and
    captured in a graph that is replayed between eager work."""
    say("layer")
    E, topk, K, I, n, rank, Tn, bits, group = 4, 2, 256, 192, 5, 8, 11, 4, 32
    rng = np.random.default_rng(3)
    wq = to_dev(synth.encode(rng.standard_normal((K, K)) * 0.05, "bf16"), "bf16")
    wg = to_dev(synth.encode(rng.standard_normal((E * 2 * I, K)) * 0.05, "bf16"), "bf16")
    wd = to_dev(synth.encode(rng.standard_normal((E * K, I)) * 0.05, "bf16"), "bf16")
    s, s2 = (f32_dev(np.exp(rng.standard_normal(c) * 0.3)) for c in (K, I))

    def state(w, s, *lead):
        codes, step, zero = T.ttq_quantize_groups(w, s, bits, group)
        return dict(s=s, codes=codes.view(*lead, -1, codes.shape[1]), scale_f16=step.view(*lead, -1, step.shape[1]),
                    zero_f16=zero.view(*lead, -1, zero.shape[1]))
    qs, gu, dn = state(wq, s), state(wg, s, E), state(wd, s2, E)
    A = to_dev(synth.encode(rng.standard_normal((n, rank, K)) / 16, "bf16"), "bf16")
    B = to_dev(synth.encode(rng.standard_normal((n, K, rank)), "bf16"), "bf16")
    router = torch.randn((K, E), device="cuda")
    ws1 = T.qgemm_adapters_workspace(Tn, K, K, bits, group, rank)
    ws2 = T.moe_workspace(Tn, topk, K, I, K, E, bits, group)
    X = torch.zeros((Tn, K), dtype=torch.bfloat16, device="cuda")
    ids = torch.zeros(Tn, dtype=torch.int32, device="cuda")

    def layer(ws1=None, ws2=None, stream=None):
        y = T.ttq_qgemm_adapters(X, qs["s"], qs["codes"], qs["scale_f16"], qs["zero_f16"], K, bits, group, A, B, ids,
                                 y_dtype=torch.bfloat16, ws=ws1, stream=stream)
        e, w = T.ttq_moe_route(y.float() @ router, topk, renormalize=True, stream=stream)
        return y, e, w, T.ttq_moe(y, e, w, gu, dn, bits, group, ws=ws2, stream=stream)

    def fill(seed):
        r = np.random.default_rng(seed)
        X.copy_(to_dev(synth.encode(r.standard_normal((Tn, K)), "bf16"), "bf16"))
        ids.copy_(i32_dev(r.integers(-1, n, Tn)))

    fill(0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer(ws1, ws2)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = layer(ws1, ws2)
    for seed in (1, 2, 3, 4):
        fill(seed)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in held]
        eager = layer()
        torch.cuda.synchronize()
        for a, b in zip(got, eager):
            assert torch.equal(a, b)
    # the experts' outputs against the definition on the library's own codes
    y, e, w, out = eager

    def numbers(q, rows, cols):
        c = host(q["codes"]).reshape(-1, cols * bits // 32)
        qn = oracle.unpack_codes(c, bits, cols).astype(np.float64).reshape(E, rows, cols)
        return (qn, *(np.repeat(host(q[k]).astype(np.float64), group, 2) for k in ("scale_f16", "zero_f16")))
    r, b = ref.moe(num(y), host(e), num(w), numbers(gu, 2 * I, K), num(s), numbers(dn, K, I), num(s2), bits, "silu", 2.0 ** -16, group)
    ref.check(num(out), r, b, False)


def test_two_calls_at_once_on_two_streams(T):
    say("two streams")
    d = moe_inputs(5, 20, 4, 2, 512, 384, 256, 4, 32, "bf16")
    ids, w = i32_dev(d["ids"]), f32_dev(d["w"])
    a = adapter_inputs(6, 20, 512, 256, 4, 16, "bf16", "mixed")
    aid = i32_dev(a["ids"])
    one = T.ttq_moe(d["X"], ids, w, d["gate_up"], d["down"], 4, 32)
    two = T.ttq_adapters_add(d["X"], a["A"], a["B"], aid)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = []
    for i in range(8):
        st = streams[i % 2]
        outs.append((T.ttq_moe(d["X"], ids, w, d["gate_up"], d["down"], 4, 32, stream=st),
                     T.ttq_adapters_add(d["X"], a["A"], a["B"], aid, stream=st)))
    torch.cuda.synchronize()
    for m, p in outs:
        assert torch.equal(m, one) and torch.equal(p, two)


def test_empty_calls(T):
    d = moe_inputs(1, 2, 3, 2, 64, 64, 32, 4, 32, "bf16")
    e = torch.empty((0, 2), dtype=torch.int32, device="cuda")
    assert T.ttq_moe(d["X"][:0], e, e.float(), d["gate_up"], d["down"], 4, 32).shape == (0, 32)
    a = adapter_inputs(6, 2, 64, 32, 4, 16, "bf16", "mixed")
    assert T.ttq_adapters_add(d["X"][:0], a["A"], a["B"], i32_dev(a["ids"])[:0]).shape == (0, 32)
    i, w = T.ttq_moe_route(torch.zeros((0, 4), device="cuda"), 2)
    assert i.shape == (0, 2) and w.shape == (0, 2)
