"""Sizes that the 8-bit products and layers take, and the first that they do not
(workspace sizes are computed on the host)."""
import os

import pytest

from conftest import ROOT

LIBPATH = os.path.join(ROOT, "online_activation_aware_amd", "libttq.so")

pytestmark = pytest.mark.skipif(not os.path.exists(LIBPATH), reason="libttq.so not built")


@pytest.fixture(scope="module")
def T():
    from online_activation_aware_amd import ttq
    ttq.lib()
    return ttq


@pytest.mark.parametrize("t,m", [(1 << 28, 16), (1 << 30, 1), (1 << 30, 256), (16, 1 << 30), (1 << 19, 1 << 19)])
def test_products_of_narrow_results(T, t, m):
    """One matrix: as many blocks of 256 x 256 as a launch can have, however they
    lie."""
    assert T.ttq_gemm_i8_workspace_bytes(t, 16, m) > 0 and T.ttq_qgemm_i8_workspace_bytes(t, 16, m) > 16 * t


@pytest.mark.parametrize("t,m", [(1 << 30, 257), (257, 1 << 30), ((1 << 19) + 1, 1 << 20)])
def test_products_beyond_one_launch(T, t, m):
    assert T.ttq_gemm_i8_workspace_bytes(t, 16, m) == 0


def test_layers_of_many_codes(T):
    """The tokens' codes are T K bytes; a token's experts share them."""
    assert T.ttq_moe_i8_workspace_bytes(1 << 14, 8, 1 << 14, 16, 16, 8) > 0
    assert T.ttq_moe_i8_workspace_bytes((1 << 17) - 1, 32, 1 << 14, 16, 16, 8) > 0
    assert T.ttq_moe_i8_workspace_bytes(1 << 17, 1, 1 << 14, 16, 16, 8) == 0
    assert T.ttq_moe_i8_workspace_bytes((1 << 24) + 1, 1, 16, 16, 16, 8) == 0
