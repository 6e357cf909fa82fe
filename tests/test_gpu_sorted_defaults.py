"""Sorted rows whose width is not a multiple of 16 bytes, in outputs that the
binding makes."""
import pytest
import torch

from gpu_util import say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def T():
    from online_activation_aware_amd import ttq
    ttq.lib()
    return ttq


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("K", [1, 3, 7, 8, 250, 1027])
@pytest.mark.parametrize("Tn,topk", [(1, 1), (1, 3), (9, 2)])
def test_defaults_of_any_width(T, dt, K, Tn, topk):
    say(f"sorted rows, default outputs {dt} K={K} T={Tn} topk={topk}")
    g = torch.Generator(device="cuda").manual_seed(K + Tn)
    pad = -(-K // 8) * 8
    X = torch.randn((Tn, pad), generator=g, device="cuda").to(dt)[:, :K]
    pos = torch.randperm(Tn * topk, generator=g, device="cuda").to(torch.int32).view(Tn, topk)
    R = T.ttq_moe_gather(X, pos)
    assert R.shape == (Tn * topk, K) and R.dtype is dt
    assert torch.equal(R[pos.long()], X[:, None].expand(-1, topk, -1))
    Y = T.ttq_moe_combine(R, pos, y_dtype=torch.float32)
    assert torch.equal(Y, topk * X.float())
    dR, dw = T.ttq_moe_combine_grad(X, R, pos)
    assert dR.shape == R.shape and dR.dtype is dt and torch.equal(dR, R)
    size = X.float().square().sum(1)
    assert torch.all((dw - size[:, None]).abs() <= 2 * K * 2.0 ** -24 * size[:, None])
    if K % 8 == 0:
        assert R.is_contiguous() and dR.is_contiguous()
