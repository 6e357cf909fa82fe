"""Refusals of the projections whose weights each token chooses, on the host
(fake, never-dereferenced device addresses) and in the binding."""
import ctypes
import os

import pytest
import torch

from conftest import ROOT

LIBPATH = os.path.join(ROOT, "online_activation_aware_amd", "libttq.so")

pytestmark = pytest.mark.skipif(not os.path.exists(LIBPATH), reason="libttq.so not built")

FAKE = 0x100000
BIG = 1 << 40


@pytest.fixture(scope="module")
def T():
    from online_activation_aware_amd import ttq
    ttq.lib()
    return ttq


def test_route(T):
    L = T.lib()

    def call(**kw):
        a = dict(l=FAKE, lt=0, T=4, E=8, ld=8, k=2, score=0, renorm=0, ids=FAKE, w=FAKE, st=None)
        a.update(kw)
        return L.ttq_moe_route(*a.values())
    for bad in (dict(E=0), dict(E=1025, ld=1025), dict(k=0), dict(k=9), dict(E=64, ld=64, k=33), dict(lt=2), dict(ld=7), dict(score=2),
                dict(score=-1), dict(l=None), dict(l=FAKE + 2), dict(lt=1, l=FAKE + 1), dict(ids=None), dict(w=None),
                dict(ids=FAKE + 1), dict(w=FAKE + 2), dict(T=-1), dict(T=(1 << 30) + 1)):
        assert call(**bad) == T.TTQ_ERR_INVALID, bad
        assert L.ttq_last_error()
    assert call(T=0, l=None, ids=None, w=None) == T.TTQ_OK


def moe_args(ttq, **kw):
    st = dict(s=FAKE, s_stride=0, codes=FAKE, scale_f16=FAKE, zero_f16=FAKE)
    gu, dn = dict(st, **kw.pop("gate_up", {})), dict(st, **kw.pop("down", {}))
    a = dict(X=FAKE, xt=1, T=4, K=256, ldx=256, ids=FAKE, w=FAKE, topk=2, E=8, I=128, M=64, gate_up=ttq.ExpertState(**gu),
             down=ttq.ExpertState(**dn), bits=4, group=32, act=0, Y=FAKE, yt=0, ldy=64)
    a.update(kw)
    return ttq.MoeArgs(**a)


def test_moe(T):
    L = T.lib()

    def call(ws=FAKE, n=BIG, **kw):
        return L.ttq_moe(ctypes.byref(moe_args(T, **kw)), ws, n, None)
    for bad in (dict(E=0), dict(E=1025), dict(topk=0), dict(topk=33), dict(K=250, ldx=256), dict(I=0), dict(I=100), dict(I=96, group=64, K=256),
                dict(bits=6), dict(group=8), dict(act=2), dict(xt=3), dict(yt=3), dict(ldx=128), dict(ldx=260), dict(ldy=63),
                dict(X=None), dict(X=FAKE + 8), dict(Y=None), dict(Y=FAKE + 2), dict(ids=None), dict(w=None), dict(ids=FAKE + 2),
                dict(gate_up=dict(s=None)), dict(gate_up=dict(s_stride=128)), dict(gate_up=dict(s_stride=258)), dict(gate_up=dict(s_stride=-4)),
                dict(down=dict(codes=None)), dict(down=dict(codes=FAKE + 4)), dict(down=dict(scale_f16=FAKE + 1)), dict(down=dict(zero_f16=None)),
                dict(M=-1), dict(T=-1), dict(ws=None), dict(ws=FAKE + 64), dict(n=64)):
        assert call(**bad) == T.TTQ_ERR_INVALID, bad
    assert call(T=1025) == T.TTQ_ERR_UNSUPPORTED
    assert call(K=1 << 16, ldx=1 << 16, I=1 << 15) == T.TTQ_ERR_UNSUPPORTED   # 2 GiB of gate and up codes
    assert L.ttq_moe(None, FAKE, BIG, None) == T.TTQ_ERR_INVALID
    assert call(T=0, X=None, ids=None, w=None, Y=None, ws=None, n=0) == T.TTQ_OK
    assert call(M=0, Y=None, ws=None, n=0) == T.TTQ_OK
    for good in ((4, 2, 256, 128, 64, 8, 4, 32), (0, 2, 256, 128, 64, 8, 4, 32), (4, 2, 256, 128, 0, 8, 4, 32), (1024, 32, 256, 32, 1, 1, 2, 16)):
        assert T.ttq_moe_workspace_bytes(*good) > 0    # an empty call's, too
    for bad in ((1025, 2, 256, 128, 64, 8, 4, 32), (4, 0, 256, 128, 64, 8, 4, 32), (4, 2, 100, 128, 64, 8, 4, 32), (4, 2, 256, 128, 64, 0, 4, 32),
                (4, 2, 256, 128, 64, 8, 7, 32)):
        assert T.ttq_moe_workspace_bytes(*bad) == 0


def adapters(ttq, **kw):
    a = dict(A=FAKE, B=FAKE, dt=1, n=4, rank=16, ranks=None, scale=None, ids=FAKE)
    a.update(kw)
    return ttq.AdaptersArgs(**a)


BAD_ADAPTERS = (dict(A=None), dict(B=None), dict(A=FAKE + 8), dict(dt=2), dict(n=-1), dict(n=65537), dict(rank=0), dict(rank=65),
                dict(ranks=FAKE + 2), dict(scale=FAKE + 1), dict(ids=None), dict(ids=FAKE + 2))


def test_adapters_add(T):
    L = T.lib()

    def call(ad=None, **kw):
        a = dict(X=FAKE, xt=1, T=4, K=256, ldx=256, ad=ctypes.byref(adapters(T, **(ad or {}))), M=64, C=FAKE, ldc=64, Y=2 * FAKE, yt=1, ldy=64,
                 ws=FAKE, n=BIG, st=None)
        a.update(kw)
        return L.ttq_adapters_add(*a.values())
    for bad in BAD_ADAPTERS:
        assert call(ad=bad) == T.TTQ_ERR_INVALID, bad
    for bad in (dict(K=250, ldx=256), dict(K=0), dict(xt=2), dict(ldx=128), dict(X=None), dict(X=FAKE + 4), dict(Y=None), dict(yt=5), dict(ldy=60),
                dict(ldc=63), dict(C=FAKE + 1), dict(C=2 * FAKE, ldc=65), dict(T=-1), dict(M=-1), dict(ws=None), dict(n=8), dict(ws=FAKE + 16)):
        assert call(**bad) == T.TTQ_ERR_INVALID, bad
    assert call(ldx=(1 << 24) + 8) == T.TTQ_ERR_UNSUPPORTED
    a = [FAKE, 1, 4, 256, 256, None, 64, FAKE, 64, FAKE, 1, 64, FAKE, BIG, None]
    assert L.ttq_adapters_add(*a) == T.TTQ_ERR_INVALID
    assert call(T=0, X=None, ad=dict(ids=None), Y=None, ws=None, n=0) == T.TTQ_OK
    assert T.ttq_adapters_workspace_bytes(4, 256, 64, 16) > 0
    for bad in ((4, 250, 64, 16), (4, 256, 64, 0), (4, 256, 64, 65), (-1, 256, 64, 16)):
        assert T.ttq_adapters_workspace_bytes(*bad) == 0


def test_qgemm_adapters(T):
    L = T.lib()

    def call(ad=None, **kw):
        a = dict(X=FAKE, xt=1, T=4, K=256, ldx=256, s=FAKE, codes=FAKE, sc=FAKE, z=FAKE, M=64, bits=4, group=32,
                 ad=ctypes.byref(adapters(T, **(ad or {}))), Y=FAKE, yt=1, ldy=64, ws=FAKE, n=BIG, st=None)
        a.update(kw)
        return L.ttq_qgemm_adapters(*a.values())
    for bad in BAD_ADAPTERS:
        assert call(ad=bad) == T.TTQ_ERR_INVALID, bad
    for bad in (dict(K=264, ldx=264), dict(bits=1), dict(group=20), dict(s=None), dict(codes=FAKE + 8), dict(sc=None), dict(z=FAKE + 1), dict(X=None),
                dict(Y=None), dict(ldy=1), dict(T=-1), dict(ws=None), dict(n=8)):
        assert call(**bad) == T.TTQ_ERR_INVALID, bad
    assert call(T=0, X=None, Y=None, ws=None, n=0) == T.TTQ_OK
    assert T.ttq_qgemm_adapters_workspace_bytes(4, 256, 64, 4, 32, 16) > 0
    for bad in ((4, 264, 64, 4, 32, 16), (4, 256, 64, 4, 32, 0), (4, 256, 64, 8, 32, 16)):
        assert T.ttq_qgemm_adapters_workspace_bytes(*bad) == 0


def test_the_binding_takes_device_tensors_only(T):
    x = torch.zeros((2, 64))
    i = torch.zeros((2, 1), dtype=torch.int32)
    for call in (lambda: T.ttq_moe_route(x, 1), lambda: T.ttq_moe(x, i, i.float(), {}, {}, 4, 32),
                 lambda: T.ttq_adapters_add(x, x[None], x[None], i[:, 0]),
                 lambda: T.ttq_qgemm_adapters(x, x, x, x, x, 4, 4, 32, x, x, i)):
        with pytest.raises(TypeError):
            call()
