"""The limits of routed_limits reject what they are meant to: no output, a
slot or some channels left out, an operand with a term or digit less, a term
of a sum missing."""
import numpy as np
import pytest

import routed_limits as lim
from test_gpu_routed import MOE
from test_gpu_routed import SHARED as SHARED_CASES

# the element-wise cases with fp32 outputs, in the form (T, E, topk, K, I, M, bits, group, xt, act, ids)
LAYERS = [(*c[:9], c[10], "any") for c in MOE] + lim.EXPERTS
LAYERS = list(dict.fromkeys(LAYERS))
SHARED = SHARED_CASES + lim.SHARED


@pytest.mark.parametrize("case", LAYERS, ids=lambda c: "-".join(map(str, c)))
def test_expert_layers(case):
    Tn, topk, I, M = case[0], case[2], case[4], case[5]
    d = lim.moe_case(case)
    y, var = lim.moe_model(d, case)
    assert lim.far(y, y, var) is None
    assert lim.far(np.zeros_like(y), y, var)
    assert lim.far(lim.moe_model(d, case, drop_slot=(Tn - 1, topk - 1))[0], y, var)
    assert lim.far(lim.moe_model(d, case, drop_channels=min(128, I // 2))[0], y, var)
    if Tn * M >= 32:                               # (one output's error may happen to be small)
        assert lim.far(lim.moe_model(d, case, less=1)[0], y, var)


@pytest.mark.parametrize("case", lim.MIXED, ids=lambda c: "-".join(map(str, c)))
def test_adapters(case):
    Tn, K, M, n, rank, xt, at = case
    d = lim.adapter_case(sum(case[:5]), *case)
    f32 = "f32" in (xt, at)
    y, var = lim.adapters(d["x"], d["a"], d["b"], d["ids"], d["ranks"], d["scale"], f32)
    assert lim.far(np.zeros_like(y), y, var)
    ids = d["ids"].copy()
    ids[np.nonzero(d["ids"] >= 0)[0][-1]] += 1     # one token with its neighbour's adapter, or none
    assert lim.far(lim.adapters(d["x"], d["a"], d["b"], ids, d["ranks"], d["scale"])[0], y, var)
    assert lim.far(lim.adapters(d["x"], d["a"], d["b"], d["ids"], d["ranks"] - 1, d["scale"])[0], y, var)
    assert lim.far(lim.adapters(d["x"], d["a"], d["b"], d["ids"], d["ranks"], d["scale"], z_terms=2)[0], y, var)
    x = d["x"].copy()
    x[:, K * 7 // 8:] = 0                          # an eighth of the channels left out
    assert lim.far(lim.adapters(x, d["a"], d["b"], d["ids"], d["ranks"], d["scale"])[0], y, var)


@pytest.mark.parametrize("case", SHARED, ids=lambda c: "-".join(map(str, c)))
def test_shared_projections(case):
    Tn, K, M, bits, group, n, rank, xt, _, _ = case
    d, num, s = lim.shared_case(case)
    y, var = lim.shared(d["x"], num, s, xt, bits, group)
    a, va = lim.adapters(d["x"], d["a"], d["b"], d["ids"], d["ranks"], d["scale"], xt == "f32")
    assert lim.far(y, y + a, var + va)
    assert lim.far(a, y + a, var + va)
    x = d["x"].copy()
    x[:, K - 32:] = 0
    assert lim.far(lim.shared(x, num, s, xt, bits, group)[0] + a, y + a, var + va)
    if xt == "f32" and (Tn > 4 or K % 128):        # x cut to two bf16 terms
        x = lim.bf16(d["x"])
        x = x + lim.bf16(d["x"] - x)
        assert lim.far(lim.shared(x, num, s, xt, bits, group)[0] + a, y + a, var + va)
