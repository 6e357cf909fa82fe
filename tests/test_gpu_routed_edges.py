"""Projections whose weights each token chooses at the ends of their ranges."""
import numpy as np
import pytest

from gpu_util import f32_dev, i32_dev, say
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
