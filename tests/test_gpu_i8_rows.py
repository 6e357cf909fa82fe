"""Rows in 8 bits whose quotients x / s lie at the ends of fp32."""
import numpy as np
import pytest
import torch

import i8_ref as ref
from gpu_util import f32_dev, host, say
from test_gpu_i8 import same

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def T():
    from online_activation_aware_amd import ttq
    ttq.lib()
    return ttq


def check(T, x, s, K):
    """The row x and the row twice, filled with ones, whole and with as many
    values as a workgroup holds or more; and one token through a projection."""
    x, s = (np.concatenate((a, np.ones(K - a.size))).astype(np.float32) for a in (x, s))
    x[len(x) // 2:] *= x[0] * np.float32(2.0 ** -30)     # of no weight beside the largest
    x[len(x) // 2:] *= s[len(x) // 2:]
    rows = np.stack((x, -x, x))
    codes, scale = T.ttq_quantize_rows(f32_dev(rows), f32_dev(s), divide=True)
    q, sc = ref.quantize(rows, s, True)
    assert np.isfinite(sc).all()
    same(scale, sc)
    np.testing.assert_array_equal(host(codes), q)


# (x, s) whose product with fp32(1 / s) is beyond fp32 and whose quotient is its largest number.
LARGEST = [("0x1.dcf94ap+127", "0x1.dcf94cp-1"), ("0x1.eafbe2p+127", "0x1.eafbe4p-1"), ("0x1.c727b4p+127", "0x1.c727b6p-1"),
           ("0x1.d3c832p+127", "0x1.d3c834p-1")]


@pytest.mark.parametrize("K", [64, 4096, 16400])
@pytest.mark.parametrize("x,s", LARGEST)
def test_quotients_of_the_largest_number(T, x, s, K):
    say(f"quantize_rows largest quotient {x} / {s} K={K}")
    x, s = float.fromhex(x), float.fromhex(s)
    assert np.float32(x) / np.float32(s) == np.finfo(np.float32).max
    with np.errstate(over="ignore"):
        assert np.isinf(np.float32(x) * (np.float32(1) / np.float32(s)))
    check(T, np.array([x, 1.0, x / 3]), np.array([s, 1.0, 1.0]), K)
    wq, ws = ref.quantize(np.random.default_rng(K).standard_normal((40, 64)))
    row = np.zeros((1, 64), np.float32)
    row[0, 5], sv = x, np.full(64, s, np.float32)
    for n in (1, 3):
        rows = np.repeat(row, n, 0)
        want = ref.product(*ref.quantize(rows, sv, True), wq, ws)
        same(T.ttq_qgemm_i8(f32_dev(rows), f32_dev(sv), torch.from_numpy(wq).cuda(), f32_dev(ws)), want)


# (x, s, the row's largest value): x / s lies next to half a step, and the remainder
# x - q s of its quotient has bits below fp32's last.
SMALL = [("0x1.046bc6p-106", "0x1.79bb8ap-40", "0x1.5e3b46p-59"), ("0x1.4b0a24p-106", "0x1.69b090p-40", "0x1.d0f38cp-59"),
         ("0x1.229e46p-106", "0x1.ed8770p-40", "0x1.2b23bap-59"), ("0x1.83755ap-106", "0x1.a0ea0cp-40", "0x1.d81bd8p-59"),
         ("0x1.6cacbcp-106", "0x1.ec386cp-40", "0x1.785d90p-59"), ("0x1.065d7ep-106", "0x1.683a74p-40", "0x1.71fde4p-59")]


@pytest.mark.parametrize("K", [64, 4096, 16400])
@pytest.mark.parametrize("x,s,top", SMALL)
def test_small_quotients_next_to_half_a_step(T, x, s, top, K):
    say(f"quantize_rows {x} / {s} beside {top} K={K}")
    x, s, top = (float.fromhex(v) for v in (x, s, top))
    assert abs(x / s / (np.float32(top) / np.float32(127)) - 0.5) < 1e-6
    xs, ss = np.full(K // 2, 0.0), np.ones(K // 2)
    xs[0], xs[1], ss[1] = top, x, s
    check(T, xs, ss, K)
