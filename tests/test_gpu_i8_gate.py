"""The gate of the 8-bit expert layer: h = act(g) u / s_down in fp32, checked to a
few roundings.

One expert whose row 0 of gate and up alone is not zero, and a down product of
one code: Y = 127^2 fp32(h / 127), rounded twice more.  g and u are whole numbers
times powers of two: exact."""
import numpy as np
import pytest
import torch

from gpu_util import f32_dev, host, i32_dev, say

pytestmark = pytest.mark.gpu

UNIT = 2.0 ** -24
STEP = 89 / 64 / 256                                   # scale of the gate: g of -87.6 to 87.6


@pytest.fixture(scope="module")
def T():
    from online_activation_aware_amd import ttq
    ttq.lib()
    return ttq


def layer(T, copies, act, u_scale, s_down, w_scale=1.0):
    """(h as Y shows it, g, u) of tokens with g = 127 c STEP for c = -127 .. 127."""
    c = np.tile(np.arange(-127, 128), copies)
    n, K, I = c.size, 16, 16
    x = np.zeros((n, K), np.float32)
    x[:, 0], x[:, 1] = 127, c                            # the row's scale is 1
    up, down = np.zeros((1, 2 * I, K), np.int8), np.zeros((1, 1, I), np.int8)
    up[0, 0, 1], up[0, I, 0], down[0, 0, 0] = 127, 1, 127
    scale = np.ones((1, 2 * I), np.float32)
    scale[0, 0], scale[0, I] = STEP, u_scale
    s = np.full((1, I), s_down, np.float32)
    dev = lambda a: torch.from_numpy(a).cuda()
    Y = T.ttq_moe_i8(f32_dev(x), i32_dev(np.zeros((n, 1))), f32_dev(np.ones((n, 1))),
                     dict(s=f32_dev(np.ones(K)), codes=dev(up), scale=f32_dev(scale)),
                     dict(s=dev(s), codes=dev(down), scale=f32_dev(np.full((1, 1), w_scale))), act=act)
    return host(Y)[:, 0].astype(np.float64), 127.0 * c * STEP, 127.0 * float(np.float32(u_scale))


def check(y, g, u, s_down, act, w_scale=1.0):
    """The roundings, in units: the exponential two (one in the last place), its sum
    with 1, the quotient, the product with u, the division by s_down, h / 127 and the
    product with the scale one each.  gelu's argument 2 sqrt(2 / pi) (g + 0.044715
    g^3): four of the cubic term, the sum's, two of the factor's, all times the
    argument."""
    arg = g if act == "silu" else 2 * np.sqrt(2 / np.pi) * (g + 0.044715 * g ** 3)
    with np.errstate(over="ignore"):
        want = 127 * w_scale * (g / (1 + np.exp(-arg))) * u / float(np.float32(s_down))
    units = 8 + (0 if act == "silu" else 7 * np.abs(arg))
    fine = np.abs(arg) < 87.7                            # behind it the exponential overflows: 0 for less than 3e-37 u
    assert fine.sum() > 20
    off = np.abs(y - want)[fine] - (units * UNIT * (1 + 1e-4) * np.abs(want))[fine]
    assert np.all(off <= 0), float((np.abs(y - want)[fine] / np.abs(want[fine] + (want[fine] == 0)) / UNIT).max())
    assert np.all(np.abs(y - want)[~fine] <= 1e-5 * np.abs(want[~fine]) + 127 * 3e-37 * u / s_down)


@pytest.mark.parametrize("copies", [1, 20])
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("s_down", [1.0, 0.7, 300.1])
def test_gate_to_a_few_roundings(T, copies, act, s_down):
    say(f"moe_i8 gate {act} copies={copies} s_down={s_down}")
    check(*layer(T, copies, act, 1.0, s_down), s_down, act)


@pytest.mark.parametrize("copies", [1, 20])
def test_gate_of_extreme_scales(T, copies):
    """s_down whose reciprocal fp32 does not hold, or not to 24 bits."""
    say(f"moe_i8 gate, extreme s_down, copies={copies}")
    for u_scale, s_down, w_scale in ((2.0 ** -100, 2.0 ** -130, 2.0 ** -20), (2.0 ** -100, 1.7 * 2.0 ** -128, 1.0), (2.0 ** 100, 1.7 * 2.0 ** 127, 1.0)):
        y, g, u = layer(T, copies, "silu", u_scale, s_down, w_scale)
        near = np.abs(g) < 10                            # act(g) u is a normal number
        check(y[near], g[near], u, s_down, "silu", w_scale)


# (a, s) whose product with fp32(1 / s) is beyond fp32 and whose quotient is its largest number.
LARGEST = [("0x1.dcf94ap+127", "0x1.dcf94cp-1"), ("0x1.eafbe2p+127", "0x1.eafbe4p-1"), ("0x1.c727b4p+127", "0x1.c727b6p-1"),
           ("0x1.d3c832p+127", "0x1.d3c834p-1")]


@pytest.mark.parametrize("a,s", LARGEST)
@pytest.mark.parametrize("n", [1, 5100])
def test_an_h_of_the_largest_number(T, a, s, n):
    """h = 64 u / s_down = fp32's largest number beside an h of 127: finite, and the
    output of a code of the small one, 0."""
    say(f"moe_i8 largest h {a} / {s} n={n}")
    a, s = np.float32(float.fromhex(a)), np.float32(float.fromhex(s))
    assert a / s == np.finfo(np.float32).max
    u_scale = next(v for k in range(-4, 5) for v in [np.float32(float(a / np.float32(64 * 127)) * (1 + k * 2.0 ** -24))] if v * np.float32(127) * np.float32(64) == a)
    x = np.zeros((n, 16), np.float32)
    x[:, 0], x[:, 1] = 127, 64
    up, down = np.zeros((1, 32, 16), np.int8), np.zeros((1, 1, 16), np.int8)
    up[0, 0, 1], up[0, 16, 0] = 1, 1                      # h of channel 0
    up[0, 1, 1], up[0, 17, 0] = 1, 1                      # and of channel 1
    down[0, 0, 1] = 127
    scale = np.ones((1, 32), np.float32)
    scale[0, 16] = u_scale
    dev = lambda v: torch.from_numpy(np.ascontiguousarray(v)).cuda()
    args = (f32_dev(x), i32_dev(np.zeros((n, 1))), f32_dev(np.ones((n, 1))), dict(s=f32_dev(np.ones(16)), codes=dev(up), scale=dev(scale)))
    Y = T.ttq_moe_i8(*args, dict(s=dev(np.full((1, 16), s)), codes=dev(down), scale=f32_dev(np.ones((1, 1)))))
    assert torch.count_nonzero(Y) == 0
    down[0, 0, 0] = 1                                     # 127 fp32(h / 127) 2^-10
    Y = T.ttq_moe_i8(*args, dict(s=dev(np.full((1, 16), s)), codes=dev(down), scale=f32_dev(np.full((1, 1), 2.0 ** -10))))
    scale = np.finfo(np.float32).max / np.float32(127)
    with np.errstate(over="ignore"):
        assert np.all(host(Y) == np.float32(127) * scale * np.float32(2.0 ** -10))
