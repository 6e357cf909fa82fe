"""Projections whose weights each token chooses at the ends of their ranges."""
import numpy as np
import pytest
import torch

import oracle
from gpu_util import f32_dev, host, i32_dev, say
from test_gpu_routed import enc, moe_inputs, num

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def T():
    from online_activation_aware_amd import ttq
    ttq.lib()
    return ttq


# ------------------------------------------------------------------ infinities of an expert layer

CODES = [(4, 32), (4, 128), (3, 16)]


@pytest.mark.parametrize("bits,group", CODES)
@pytest.mark.parametrize("xt", ["bf16", "f32"])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("Tn", [1, 2, 12])
def test_moe_infinite_x(T, Tn, sign, xt, bits, group):
    say(f"moe inf x {sign} {xt} b{bits} g{group} T={Tn}")
    d = moe_inputs(Tn, Tn, 2, 2, 256, 256, 40, bits, group, xt)
    args = i32_dev(d["ids"]), f32_dev(d["w"]), d["gate_up"], d["down"], bits, group
    want = num(T.ttq_moe(d["X"], *args))
    X = d["X"].clone()
    X[0, 77] = sign * np.inf
    y = num(T.ttq_moe(X, *args))
    assert np.all(np.isnan(y[0]))
    np.testing.assert_array_equal(y[1:], want[1:])


@pytest.mark.parametrize("bits,group", CODES)
@pytest.mark.parametrize("xt", ["bf16", "f32"])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("Tn", [1, 2, 12])
def test_moe_overflowing_h(T, Tn, sign, xt, bits, group):
    """Expert 0, of token 0 alone, has one channel of h beyond fp32 (its s_down is 2^-126)."""
    say(f"moe inf h {sign} {xt} b{bits} g{group} T={Tn}")
    K, I, M = 256, 256, 40
    d = moe_inputs(Tn + 50, Tn, 2, 1, K, I, M, bits, group, xt)
    d["ids"][:] = 1
    d["ids"][0] = 0
    w = d["w"] + 1
    x = d["x"] * 2.0 ** 10                         # exact; |g| and |u| of hundreds
    X = enc(x, xt)[0]
    n, s_in = d["gate_up_ref"]
    q, dl, z = (v[0] for v in n)
    gu = (x[0] / s_in) @ ((q - z) * dl).T
    h = gu[:I] / (1 + np.exp(-np.clip(gu[:I], -700, 700))) * gu[I:]
    c = int(np.argmax(h * sign))
    assert h[c] * sign > 1000                      # times 2^126 and a weight above 1: beyond fp32
    args = i32_dev(d["ids"]), f32_dev(w), d["gate_up"]
    want = num(T.ttq_moe(X, *args, d["down"], bits, group))
    assert np.all(np.isfinite(want))
    s = d["down"]["s"].clone()
    s[0, c] = 2.0 ** -126
    y = num(T.ttq_moe(X, *args, dict(d["down"], s=s), bits, group))
    assert np.all(np.isnan(y[0]))
    np.testing.assert_array_equal(y[1:], want[1:])


# ------------------------------------------------------------------ values next to zero

@pytest.mark.parametrize("g", [2.0, 0.5, -1.0, -3.0, -4.0, -5.5])
@pytest.mark.parametrize("act", ["gelu", "silu"])
@pytest.mark.parametrize("xt", ["bf16", "f32"])
@pytest.mark.parametrize("Tn", [1, 5])
def test_moe_activation_keeps_its_precision(T, Tn, xt, act, g):
    """Every gate is g, every up value 1 and the second product passes h on: y is the activation of g itself."""
    say(f"moe act {act} {xt} g={g} T={Tn}")
    K = I = M = 32
    q = np.full((2 * I, K), 8)
    q[:, 0] = 9                                    # (9 - 8) step times x[0] = 1
    step = np.repeat([abs(g), 1.0], I)[:, None].astype(np.float16)
    if g < 0:
        q[:I, 0] = 7
    qd = np.full((M, I), 8) + np.eye(I, dtype=int)

    def state(q, step):
        return dict(s=torch.ones(32, device="cuda"), codes=i32_dev(oracle.pack_codes(q, 4))[None],
                    scale_f16=torch.from_numpy(step).cuda()[None], zero_f16=torch.full((1, len(q), 1), 8.0, dtype=torch.float16, device="cuda"))
    x = np.zeros((Tn, K))
    x[:, 0] = 1
    y = num(T.ttq_moe(enc(x, xt)[0], torch.zeros((Tn, 1), dtype=torch.int32, device="cuda"), torch.ones((Tn, 1), device="cuda"),
                      state(q, step), state(qd, np.ones((M, 1), np.float16)), 4, 32, act=act))
    u = np.sqrt(2 / np.pi) * (g + 0.044715 * g ** 3)
    want = g / (1 + np.exp(-g)) if act == "silu" else g / (1 + np.exp(-2 * u))
    # g off by 8 roundings moves the value by its slope over it, at most 1 + |g| (silu), 1 + 2 u' |g| (gelu); the exponential's
    # argument by 4 roundings of itself; 16 more roundings; h as digits (half a scale and 3 roundings) or terms
    slope = 1 + abs(g) * (1 if act == "silu" else 2 * np.sqrt(2 / np.pi) * (1 + 3 * 0.044715 * g * g))
    rel = 2.0 ** -24 * (8 * slope + 4 * abs(2 * u) + 16)
    if Tn == 1:
        rel += 2.0 ** -19 if xt == "bf16" else 2.0 ** -23
    else:
        # the second product is a difference, y = P - 24 S, of P = sum (16 + q) h = 31 * 24 h + 25 h = 769 h and S = 32 h.  P in four
        # steps of at most P/4, P/2, 3 P/4 and P in size: 2.5 roundings of 2^-23 P; S in 31 additions of 2^-24: 15.5; the zero
        # term and the running sum 3: 21 * 769 * 2^-23 < 2^-9
        rel += 2.0 ** -9
    assert np.all(np.abs(y - want) <= rel * abs(want)), (y[0, 0], want, rel)


@pytest.mark.parametrize("lt", ["f32", "bf16"])
def test_route_small_sigmoid_scores(T, lt):
    """Scores below fp32's range: renormalized, their ratios are weights as any others."""
    say(f"route small sigmoids {lt}")
    rows = [[-80, -81, -82.5, -90, -95], [-89, -90, -91, -89.5, -300], [-95, -95, -96, -97, -95], [-200, -201, -199, -200, -205],
            [-744, -743, -744, -742, -741], [0.5, -100, -200, -1, 3], [-3e38, -1e38, -2e38, -3e38, -1e38]]
    L, x = enc(rows, lt)
    for topk in (1, 3):
        ids, w = T.ttq_moe_route(L, topk, score="sigmoid", renormalize=True)
        order = np.argsort(-x, axis=1, kind="stable")[:, :topk]
        np.testing.assert_array_equal(host(ids), order)
        v = np.take_along_axis(x, order, 1)
        r = np.exp(np.minimum(v, 0) - np.minimum(v[:, :1], 0)) / (1 + np.exp(-np.abs(v)))
        r[v[:, 0] < -745] = 0                      # no score left, in 64 bits either
        r /= np.maximum(r.sum(1, keepdims=True), 1e-300)
        # the exponential of a difference up to 100, in fp32, and 8 roundings, of the score and of the sum
        assert np.all(np.abs(num(w) - r) <= 2.0 ** -24 * 2 * (100 + 8 + topk) * r + 1e-37), (num(w), r)
    ids, w = T.ttq_moe_route(L, 5, score="sigmoid")
    v = np.take_along_axis(x, host(ids), 1)
    with np.errstate(over="ignore"):
        r = 1 / (1 + np.exp(-v))
    # 2^-149 is the least fp32 number: half a step of it besides the relative error
    assert np.all(np.abs(num(w) - r) <= (np.abs(v).clip(max=104) + 10) * 2.0 ** -23 * r + 2.0 ** -149)


# ------------------------------------------------------------------ shared memory

@pytest.mark.parametrize("Tn", [1, 5, 130])
@pytest.mark.parametrize("add", [False, True])
def test_adapters_written_over_x(T, Tn, add):
    """Y may lie on X, alone or as C too: a residual connection in place."""
    say(f"adapters over X T={Tn} add={add}")
    rng = np.random.default_rng(Tn)
    K, rank, n = 4096, 16, 3
    A, B = enc(rng.standard_normal((n, rank, K)) / 64, "bf16")[0], enc(rng.standard_normal((n, K, rank)), "bf16")[0]
    ids = i32_dev(rng.integers(0, n, Tn))
    for _ in range(4):
        X = enc(rng.standard_normal((Tn, K)), "bf16")[0]
        want = T.ttq_adapters_add(X, A, B, ids, C=X if add else None, y_dtype=torch.bfloat16)
        Z = X.clone()
        T.ttq_adapters_add(Z, A, B, ids, C=Z if add else None, Y=Z)
        # one token in place takes two launches, whose sums have another order: each within 64 + 16 fp32 roundings, then bf16
        got, r = num(Z), num(want)
        x = num(X)
        mag = np.zeros_like(r)
        for t in range(Tn):
            a = int(ids[t])
            mag[t] = np.abs(num(B)[a]) @ (np.abs(num(A)[a]) @ np.abs(x[t]))
        assert np.all(np.abs(got - r) <= 2.0 ** -7 * np.abs(r) + 2 * (K + 2 * rank) * 2.0 ** -23 * mag)


# ------------------------------------------------------------------ calling

def test_calls_by_name_and_with_a_stream_in_place(T):
    say("calls by name")
    d = moe_inputs(4, 3, 2, 2, 64, 64, 32, 4, 32, "bf16")
    L = torch.randn((3, 4), device="cuda")
    ids, w = T.ttq_moe_route(L, 2)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    for i2, w2 in (T.ttq_moe_route(logits=L, topk=2), T.ttq_moe_route(L, 2, "softmax", False, None, None, st),
                   T.ttq_moe_route(L, 2, stream=st.cuda_stream)):
        torch.cuda.synchronize()
        assert torch.equal(ids, i2) and torch.equal(w, w2)
    args = dict(X=d["X"], ids=i32_dev(d["ids"]), w=f32_dev(d["w"]), gate_up=d["gate_up"], down=d["down"], bits=4, group=32)
    assert torch.equal(T.ttq_moe(**args), T.ttq_moe(*args.values()))


def test_refused_sizes_allocate_nothing(T):
    say("refused sizes")
    L = torch.zeros((4, 8), device="cuda")
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.memory_allocated()
    for topk in (0, 9, -1, 1 << 20):
        with pytest.raises(T.TTQError):
            T.ttq_moe_route(L, topk)
    assert torch.cuda.max_memory_allocated() - before < 1 << 16


@pytest.mark.parametrize("xt", ["f32", "bf16"])
def test_two_captured_graphs(T, xt):
    """An expert layer and a shared projection in a graph each, with workspaces of their own, replayed in turn with
    eager calls between."""
    say(f"graphs {xt}")
    Tn, K, I, n, rank, dt = 20, 640, 512, 4, 8, {"f32": torch.float32, "bf16": torch.bfloat16}[xt]
    d = moe_inputs(3, Tn, 3, 2, K, I, K, 4, 64, xt)
    ids, w = i32_dev(d["ids"]), f32_dev(d["w"])
    q = {k: v[0].contiguous() for k, v in d["gate_up"].items() if k != "s"}
    s, M = d["gate_up"]["s"], 2 * I
    rng = np.random.default_rng(1)
    A, B = enc(rng.standard_normal((n, rank, K)) / 16, xt)[0], enc(rng.standard_normal((n, M, rank)), xt)[0]
    X, aid = torch.zeros((Tn, K), dtype=dt, device="cuda"), torch.zeros(Tn, dtype=torch.int32, device="cuda")

    def layer(ws=None):
        return T.ttq_moe(X, ids, w, d["gate_up"], d["down"], 4, 64, ws=ws)

    def shared(ws=None):
        return T.ttq_qgemm_adapters(X, s, q["codes"], q["scale_f16"], q["zero_f16"], M, 4, 64, A, B, aid, ws=ws)
    own = [T.moe_workspace(Tn, 2, K, I, K, 3, 4, 64), T.qgemm_adapters_workspace(Tn, K, M, 4, 64, rank)]
    graphs, held = [], []
    for call, ws in zip((layer, shared), own):
        call(ws)
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            held.append(call(ws))
    for seed in range(4):
        r = np.random.default_rng(seed)
        X.copy_(enc(r.standard_normal((Tn, K)), xt)[0])
        aid.copy_(i32_dev(r.integers(-1, n, Tn)))
        for i in (seed % 2, 1 - seed % 2):
            graphs[i].replay()
        got = [h.clone() for h in held]
        eager = layer(), shared()
        torch.cuda.synchronize()
        for a, b in zip(got, eager):
            assert torch.equal(a, b)
