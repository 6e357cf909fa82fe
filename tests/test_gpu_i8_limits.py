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


@pytest.mark.parametrize("per", [False, True])
def test_a_layer_whose_slots_have_more_than_2_gib_of_codes(T, per):
    """Every token's result is that of a call of 64 tokens."""
    say(f"moe_i8 2 GiB of codes, scales per expert: {per}")
    Tn, topk, K, I, M, E = 1 << 14, 9, 1 << 14, 48, 20, 4
    assert Tn * topk * K > 1 << 31
    g = torch.Generator(device="cuda").manual_seed(3)
    rand = lambda *shape: torch.rand(shape, generator=g, device="cuda")
    X = torch.randn((Tn, K), generator=g, device="cuda").bfloat16()
    ids = torch.randint(0, E, (Tn, topk), generator=g, device="cuda", dtype=torch.int32)
    w = rand(Tn, topk) + 0.1
    up = dict(s=(rand(E, K) if per else rand(K)) + 0.5, codes=codes_like(g, E, 2 * I, K), scale=(rand(E, 2 * I) + 0.5) * (0.02 / K ** 0.5))
    down = dict(s=rand(E, I) + 0.5, codes=codes_like(g, E, M, I), scale=(rand(E, M) + 0.5) * (0.02 / I ** 0.5))
    Y = T.ttq_moe_i8(X, ids, w, up, down)
    assert torch.isfinite(Y).all()
    for lo in (0, 64, Tn // 2, Tn - 64):
        part = T.ttq_moe_i8(X[lo:lo + 64], ids[lo:lo + 64].contiguous(), w[lo:lo + 64].contiguous(), up, down)
        assert torch.equal(part, Y[lo:lo + 64]), lo


def test_a_layer_of_just_under_2_gib_of_codes(T):
    say("moe_i8 just under 2 GiB")
    Tn, topk, K, I, M, E = (1 << 17) - 1, 2, 1 << 14, 16, 8, 2
    g = torch.Generator(device="cuda").manual_seed(4)
    rand = lambda *shape: torch.rand(shape, generator=g, device="cuda")
    X = torch.randn((Tn, K), generator=g, device="cuda", dtype=torch.bfloat16)
    ids = torch.randint(0, E, (Tn, topk), generator=g, device="cuda", dtype=torch.int32)
    w = rand(Tn, topk) + 0.1
    up = dict(s=rand(K) + 0.5, codes=codes_like(g, E, 2 * I, K), scale=(rand(E, 2 * I) + 0.5) * (0.02 / K ** 0.5))
    down = dict(s=rand(E, I) + 0.5, codes=codes_like(g, E, M, I), scale=(rand(E, M) + 0.5) * (0.02 / I ** 0.5))
    Y = T.ttq_moe_i8(X, ids, w, up, down)
    assert torch.isfinite(Y).all()
    for lo in (0, Tn // 2, Tn - 64):
        part = T.ttq_moe_i8(X[lo:lo + 64], ids[lo:lo + 64].contiguous(), w[lo:lo + 64].contiguous(), up, down)
        assert torch.equal(part, Y[lo:lo + 64]), lo
