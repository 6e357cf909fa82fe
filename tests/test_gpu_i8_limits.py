"""8-bit products and layers at the largest sizes that they take."""
import pytest
import torch

from gpu_util import say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def T():
    from online_activation_aware_amd import ttq
    ttq.lib()
    return ttq


def codes_like(g, *shape):
    return torch.randint(-127, 128, shape, generator=g, device="cuda", dtype=torch.int8)


@pytest.mark.parametrize("Tn,M", [((1 << 28) + 3, 17), (17, (1 << 28) + 3)])
def test_long_and_narrow_products(T, Tn, M):
    """Y of 2^32 values and more; the results of rows at both ends, around 2^32 bytes
    and in between."""
    say(f"gemm_i8 T={Tn} M={M}")
    g = torch.Generator(device="cuda").manual_seed(5)
    x, w = codes_like(g, Tn, 16), codes_like(g, M, 16)
    xs, ws = torch.rand(Tn, generator=g, device="cuda"), torch.rand(M, generator=g, device="cuda")
    Y = T.ttq_gemm_i8(x, xs, w, ws, y_dtype=torch.bfloat16)
    n = max(Tn, M)
    at = torch.cat([torch.tensor([0, 1, n - 260, n - 4, n - 3, n - 2, n - 1], device="cuda"), torch.randint(0, n, (100000,), generator=g, device="cuda")])
    x, xs, got = (x[at], xs[at], Y[at]) if Tn > M else (x, xs, Y)
    w, ws, got = (w[at], ws[at], Y[:, at]) if M > Tn else (w, ws, got)
    sums = x.float() @ w.float().t().contiguous()        # whole numbers below 2^24
    assert torch.equal(got, (sums * xs[:, None] * ws[None, :]).bfloat16())
