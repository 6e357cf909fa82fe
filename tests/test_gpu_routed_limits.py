"""Projections whose weights each token chooses against fp64, within the
variance of their rounding errors (routed_limits): outputs that miss a slot, a
slice of channels or a term of an operand are rejected, see
test_routed_limits.py."""
import numpy as np
import pytest
import torch

import routed_limits as lim
import routed_ref as ref
from gpu_util import f32_dev, i32_dev, say, to_dev
from online_activation_aware_amd import synth
from test_gpu_routed import num
from test_routed_limits import LAYERS, SHARED

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def T():
    from online_activation_aware_amd import ttq
    ttq.lib()
    return ttq


def dev(a, dt):
    return to_dev(synth.encode(np.asarray(a, np.float64), dt), dt)


def state_dev(q):
    return dict(s=f32_dev(q["s"]), codes=i32_dev(q["codes"]), scale_f16=torch.from_numpy(q["step"]).cuda(),
                zero_f16=torch.from_numpy(q["zero"]).cuda())


def moe_call(T, d, case, a=0, b=None):
    bits, group, xt, act = case[6:10]
    b = len(d["ids"]) if b is None else b
    gu, dn = d.setdefault("dev", [state_dev(d["gate_up"]), state_dev(d["down"])])
    return num(T.ttq_moe(dev(d["x"][a:b], xt), i32_dev(d["ids"][a:b]), f32_dev(d["w"][a:b]), gu, dn, bits, group, act=act))


# ------------------------------------------------------------------ experts

@pytest.mark.parametrize("case", LAYERS, ids=lambda c: "-".join(map(str, c)))
def test_expert_layers(T, case):
    say(f"layer {case}")
    d = lim.moe_case(case)
    y, var = lim.moe_model(d, case)
    got = moe_call(T, d, case)
    lim.check(got, y, var)
    np.testing.assert_array_equal(moe_call(T, d, case), got)


@pytest.mark.parametrize("xt", ["bf16", "f32"])
@pytest.mark.parametrize("bits,group", [(4, 32), (4, 128), (3, 16)])
def test_a_token_in_calls_of_other_sizes(T, bits, group, xt):
    """Calls that hold x / s and h alike (one and two tokens; three and more) give a token the same outputs up to
    the order of fp32 sums, others up to their operands' errors."""
    say(f"layer in parts b{bits} g{group} {xt}")
    case = (24, 4, 2, 384, 2304, 96, bits, group, xt, "silu", "any")
    d = lim.moe_case(case)
    whole = moe_call(T, d, case)
    y, sums = lim.moe_model(d, case, own=False)
    full = lim.moe_model(d, case)[1]

    def part(a, b):
        rows = dict(d, **{k: d[k][a:b] for k in ("x", "ids", "w")})
        own, v = (lim.moe_model(rows, (b - a, *case[1:]), own=o)[1] for o in (True, False))
        return moe_call(T, d, case, a, b), own, v
    digits = bits == 4 and group >= 32
    for a, b in ((0, 3), (4, 12), (7, 24)):
        got, _, v = part(a, b)
        lim.check(got, whole[a:b], v + sums[a:b])
    for a in (0, 9, 22):
        one, own, v = part(a, a + 1)
        two, _, v2 = part(a, a + 2)
        lim.check(one, two[:1], v + v2[:1])
        lim.check(one, whole[a:a + 1], own + full[a:a + 1] if digits else v + sums[a:a + 1])


# ------------------------------------------------------------------ adapters

@pytest.mark.parametrize("yt", ["f32", "bf16"])
@pytest.mark.parametrize("case", lim.MIXED + lim.RUNS, ids=lambda c: "-".join(map(str, c)))
def test_adapters_in_any_order(T, case, yt):
    say(f"adapters {case} {yt}")
    Tn, K, M, n, rank, xt, at = case
    d = lim.adapter_case(sum(case[:5]), *case, runs=case in lim.RUNS)
    none = d["ids"] < 0
    assert none.any() and (len(set(d["ids"][:32])) > 5) == (case in lim.MIXED)
    y, var = lim.adapters(d["x"], d["a"], d["b"], d["ids"], d["ranks"], d["scale"], "f32" in (xt, at))
    A, B = dev(d["a"], at), dev(d["b"], at)
    for i, r in enumerate(d["ranks"]):             # what lies behind a rank is not used
        A[i, r:] = float("nan")
        B[i, :, r:] = float("nan")
    X, args = dev(d["x"], xt), (A, B, i32_dev(d["ids"]))
    kw = dict(ranks=i32_dev(d["ranks"]), scale=f32_dev(d["scale"]))
    got = num(T.ttq_adapters_add(X, *args, **kw))
    lim.check(got, y, var + (lim.U * y) ** 2)
    assert np.all(got[none] == 0)
    C = dev(d["rng"].standard_normal((Tn, M)), yt)
    c = num(C)
    out = T.ttq_adapters_add(X, *args, C=C, **kw)
    half = 2.0 ** -8 if yt == "bf16" else lim.U
    lim.check(num(out), c + y, var + (half * (c + y)) ** 2)
    np.testing.assert_array_equal(num(out)[none], c[none])
    assert torch.equal(T.ttq_adapters_add(X, *args, C=C, Y=C, **kw), out)


# ------------------------------------------------------------------ a shared projection with adapters

@pytest.mark.parametrize("case", SHARED, ids=lambda c: "-".join(map(str, c)))
def test_shared_projections(T, case):
    """Against fp64, and against the two calls it stands for up to the order of fp32 sums (and their bits of fp32 X)."""
    say(f"shared {case}")
    Tn, K, M, bits, group, n, rank, xt, _, _ = case
    d, nums, s = lim.shared_case(case)
    y, var = lim.shared(d["x"], nums, s, xt, bits, group)
    a, va = lim.adapters(d["x"], d["a"], d["b"], d["ids"], d["ranks"], d["scale"], xt == "f32")
    q = state_dev(d["state"])
    X, state = dev(d["x"], xt), (q["s"], q["codes"], q["scale_f16"], q["zero_f16"], M, bits, group)
    ad = dict(A=dev(d["a"], xt), B=dev(d["b"], xt), ids=i32_dev(d["ids"]), ranks=i32_dev(d["ranks"]), scale=f32_dev(d["scale"]))
    got = num(T.ttq_qgemm_adapters(X, *state, **ad))
    lim.check(got, y + a, var + va)
    ws = T.workspace(Tn, K, M, bits, group)
    two = num(T.ttq_adapters_add(X, C=T.ttq_qgemm(X, *state, ws=ws), **ad))
    qn, dl, z = nums
    R = d["x"] ** 2 @ (((qn - z) * dl / s) ** 2).T
    # ttq_qgemm keeps 16 bits of fp32 x and of the weight for more than four tokens (their product's last part left out: 2^-14)
    half = 2.0 ** -14 if xt == "f32" and (Tn > 4 or K % 128) else 0.0
    lim.check(got, two, lim.U ** 2 * (16 * R + 4 * y ** 2 + 4 * a ** 2) + half ** 2 / 3 * R)


# ------------------------------------------------------------------ memory around a call

@pytest.mark.parametrize("case", [(1, 3, 2, 544, 1056, 65, 4, 32, "bf16", "silu", "any"), (2, 4, 2, 640, 384, 129, 4, 128, "f32", "gelu", "any"),
                                  (5, 3, 2, 96, 160, 33, 4, 32, "bf16", "gelu", "any"), (20, 2, 2, 640, 2432, 33, 4, 128, "bf16", "silu", "any"),
                                  (18, 5, 2, 512, 640, 70, 4, 64, "f32", "silu", "any"), (9, 3, 2, 96, 96, 34, 3, 16, "bf16", "silu", "any")],
                         ids=lambda c: "-".join(map(str, c)))
def test_expert_layer_steps_at_half_words_and_a_used_workspace(T, case):
    """Steps and zeros whose arrays start within a word (each, or one of them), a workspace full of NaN, and nothing
    written behind it or beside Y."""
    say(f"layer memory {case}")
    Tn, E, topk, K, I, M, bits, group, xt, act, _ = case
    d = lim.moe_case(case)
    rng = np.random.default_rng(1)
    d["ids"] = np.argsort(rng.random((Tn, E)), axis=1)[:, :topk].astype(np.int32)
    y, var = lim.moe_model(d, case)
    need = T.ttq_moe_workspace_bytes(Tn, topk, K, I, M, E, bits, group)
    for by in ((1, 1), (1, 0), (0, 1)):
        def place(q):
            st = state_dev(q)
            for k, n in zip(("scale_f16", "zero_f16"), by):
                buf = torch.full((st[k].numel() + 2,), float("nan"), dtype=torch.float16, device="cuda")
                st[k] = buf[n:n + st[k].numel()].view(st[k].shape).copy_(st[k])
            return st
        ws = torch.full((need + 512,), 255, dtype=torch.uint8, device="cuda")
        Y = torch.full((Tn + 2, M + 3), -7.0, device="cuda")
        T.ttq_moe(dev(d["x"], xt), i32_dev(d["ids"]), f32_dev(d["w"]), place(d["gate_up"]), place(d["down"]), bits, group, act=act,
                  Y=Y[1:-1, 1:1 + M], ws=ws[:need])
        got = num(Y)
        lim.check(got[1:-1, 1:1 + M], y, var)
        assert np.all(got[[0, -1]] == -7) and np.all(got[:, 0] == -7) and np.all(got[:, 1 + M:] == -7)
        assert torch.all(ws[need:] == 255)


@pytest.mark.parametrize("xt", ["bf16", "f32"])
@pytest.mark.parametrize("bits,group", [(4, 32), (4, 64), (4, 128), (3, 16), (2, 32)])
@pytest.mark.parametrize("Tn", [1, 2, 5, 40])
def test_zeros_of_any_value(T, Tn, bits, group, xt):
    """Zeros between the codes, below and far above them are taken as they are."""
    say(f"layer zeros b{bits} g{group} {xt} T={Tn}")
    case = (Tn, 3, 2, 384, 256, 70, bits, group, xt, "silu", "any")
    d = lim.moe_case(case)
    rng = np.random.default_rng(Tn)
    d["ids"] = np.argsort(rng.random((Tn, 3)), axis=1)[:, :2].astype(np.int32)
    for q in (d["gate_up"], d["down"]):
        z = (rng.integers(-4, 20, q["zero"].shape) + rng.integers(0, 8, q["zero"].shape) / 8).astype(np.float16)
        z[rng.random(z.shape) < 0.02] = 200.125
        q["zero"] = z
        q["num"] = (*q["num"][:2], np.repeat(z.astype(np.float64), group, 2))
    d["x"] = np.round(d["x"] * 8) / 1024
    # Weights of one sign: the roundings of a group's sum of x / s are common to all of a token's outputs, not independent
    # as in the variances, so the limit is the sum of the largest roundings.
    gu, dn = d["gate_up"], d["down"]
    y, b = ref.moe(d["x"], d["ids"], d["w"].astype(np.float64), gu["num"], gu["s"].astype(np.float64), dn["num"], dn["s"].astype(np.float64),
                   bits, "silu", 2.0 ** -16 if xt == "bf16" else 2.0 ** -23, group)
    ref.check(moe_call(T, d, case), y, b, False)


def test_shared_projection_of_more_codes_than_a_buffer_holds(T):
    """fp32 X on a weight of 2 GiB of codes: rows on both sides of where the calls inside part them."""
    say("shared 2 GiB")
    Tn, K, M, group = 5, 65536, 65600, 32
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    codes = torch.randint(-2 ** 31, 2 ** 31 - 1, (M, K // 8), dtype=torch.int32, device="cuda", generator=g)
    step = torch.rand((M, K // group), device="cuda", generator=g).add_(0.5).mul_(0.01).half()
    zero = torch.randint(0, 16, (M, K // group), device="cuda", generator=g).half()
    X, s = torch.randn((Tn, K), device="cuda", generator=g), torch.rand(K, device="cuda", generator=g) + 0.5
    A, B = torch.zeros((1, 4, K), device="cuda"), torch.zeros((1, M, 4), device="cuda")
    y = T.ttq_qgemm_adapters(X, s, codes, step, zero, M, 4, group, A, B, torch.zeros(Tn, dtype=torch.int32, device="cuda"))
    rows = torch.tensor([0, 32767, 65503, 65504, 65535, 65536, 65599], device="cuda")
    c = codes[rows].view(torch.uint8)
    q = num(torch.stack((c & 15, c >> 4), -1).flatten(-2).float())
    d, z = (np.repeat(num(t[rows].float()), group, 1) for t in (step, zero))
    r, var = lim.shared(num(X), (q, d, z), num(s), "f32", 4, group)
    lim.check(num(y[:, rows]), r, var)
