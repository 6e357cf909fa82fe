"""The binding of the projections whose weights each token chooses: its first
argument by name."""
import os

import pytest
import torch

from conftest import ROOT

pytestmark = pytest.mark.skipif(not os.path.exists(os.path.join(ROOT, "online_activation_aware_amd", "libttq.so")),
                                reason="libttq.so not built")


def test_the_first_argument_by_name():
    from online_activation_aware_amd import ttq
    x = torch.zeros((2, 64))
    with pytest.raises(TypeError, match="device tensor"):
        ttq.ttq_moe_route(logits=x, topk=1)
    with pytest.raises(TypeError, match="device tensor"):
        ttq.ttq_moe(ids=x, w=x, X=x, gate_up={}, down={}, bits=4, group=32)
    for call in (ttq.ttq_moe_route, ttq.ttq_adapters_add):
        with pytest.raises(TypeError, match="argument"):
            call(topk=1)
