"""Refusals of the 8-bit layers and of the sorted rows, on the host (fake,
never-dereferenced device addresses) and in the binding."""
import ctypes
import os

import pytest
import torch

from conftest import ROOT

LIBPATH = os.path.join(ROOT, "online_activation_aware_amd", "libttq.so")

pytestmark = pytest.mark.skipif(not os.path.exists(LIBPATH), reason="libttq.so not built")

FAKE = 0x100000
BIG = 1 << 50


@pytest.fixture(scope="module")
def T():
    from online_activation_aware_amd import ttq
    ttq.lib()
    return ttq


def refuses(T, fn, ok, bad, unsupported=()):
    for kw in bad:
        assert fn(*dict(ok, **kw).values()) == T.TTQ_ERR_INVALID, kw
        assert T.lib().ttq_last_error()
    for kw in unsupported:
        assert fn(*dict(ok, **kw).values()) == T.TTQ_ERR_UNSUPPORTED, kw


def test_quantize_rows(T):
    fn = T.lib().ttq_quantize_rows
    ok = dict(X=FAKE, xt=1, R=4, K=256, ldx=256, s=FAKE, div=1, q=FAKE, ldc=256, scale=FAKE, st=None)
    refuses(T, fn, ok, (dict(K=0), dict(K=-16), dict(K=24), dict(K=(1 << 17) + 16, ldx=1 << 18, ldc=1 << 18), dict(xt=2), dict(ldx=248), dict(ldx=260),
                        dict(X=None), dict(X=FAKE + 8), dict(s=FAKE + 4), dict(q=None), dict(q=FAKE + 8), dict(ldc=240), dict(ldc=264),
                        dict(scale=None), dict(scale=FAKE + 2), dict(R=-1), dict(R=(1 << 30) + 1)))
    assert fn(*dict(ok, R=0, X=None, q=None, scale=None).values()) == T.TTQ_OK


def test_gemm(T):
    fn = T.lib().ttq_gemm_i8
    ok = dict(X=FAKE, xs=FAKE, T=4, K=256, ldx=256, W=FAKE, ws=FAKE, M=64, ldw=256, Y=FAKE, yt=0, ldy=64, wsp=FAKE, n=BIG, st=None)
    refuses(T, fn, ok, (dict(K=0), dict(K=40), dict(K=1 << 18, ldx=1 << 18, ldw=1 << 18), dict(X=None), dict(X=FAKE + 1), dict(ldx=255), dict(ldx=264),
                        dict(xs=None), dict(xs=FAKE + 1), dict(W=None), dict(W=FAKE + 4), dict(ldw=128), dict(ldw=257), dict(ws=None), dict(ws=FAKE + 2),
                        dict(Y=None), dict(Y=FAKE + 2), dict(yt=2), dict(ldy=63), dict(T=-1), dict(M=-1), dict(wsp=None), dict(wsp=FAKE + 16), dict(n=8)),
            (dict(ldx=(1 << 22) + 16), dict(ldw=(1 << 22) + 16), dict(T=1 << 30, M=1 << 30, ldy=1 << 30)))
    assert fn(*dict(ok, T=0, X=None, xs=None, W=None, ws=None, Y=None, wsp=None).values()) == T.TTQ_OK
    assert fn(*dict(ok, M=0, X=None, xs=None, W=None, ws=None, Y=None, wsp=None).values()) == T.TTQ_OK
    assert T.ttq_gemm_i8_workspace_bytes(4, 256, 64) > 0 and T.ttq_gemm_i8_workspace_bytes(0, 256, 0) > 0
    for bad in ((-1, 256, 64), (4, 250, 64), (4, 0, 64), (4, 1 << 18, 64), (4, 256, -1)):
        assert T.ttq_gemm_i8_workspace_bytes(*bad) == 0 and T.ttq_qgemm_i8_workspace_bytes(*bad) == 0


def test_qgemm(T):
    fn = T.lib().ttq_qgemm_i8
    ok = dict(X=FAKE, xt=1, T=4, K=256, ldx=256, s=FAKE, W=FAKE, ws=FAKE, M=64, ldw=256, Y=FAKE, yt=0, ldy=64, wsp=FAKE, n=BIG, st=None)
    refuses(T, fn, ok, (dict(K=0), dict(K=40), dict(X=None), dict(X=FAKE + 4), dict(xt=2), dict(ldx=248), dict(ldx=258), dict(s=FAKE + 8), dict(W=None),
                        dict(ldw=128), dict(ws=None), dict(Y=None), dict(yt=3), dict(ldy=60), dict(T=-1), dict(wsp=None), dict(n=1024)),
            (dict(ldw=(1 << 22) + 16),))
    assert fn(*dict(ok, T=0, X=None, W=None, ws=None, Y=None, wsp=None).values()) == T.TTQ_OK
    assert T.ttq_qgemm_i8_workspace_bytes(4, 256, 64) >= 4 * 256 + 4 * 4


def test_sort(T):
    fn = T.lib().ttq_moe_sort
    ok = dict(ids=FAKE, T=4, topk=2, E=8, off=FAKE, order=FAKE, pos=FAKE, wsp=FAKE, n=BIG, st=None)
    refuses(T, fn, ok, (dict(topk=0), dict(topk=33), dict(E=0), dict(E=1025), dict(T=-1), dict(T=1 << 30), dict(ids=None), dict(ids=FAKE + 2),
                        dict(off=None), dict(order=None), dict(pos=FAKE + 1), dict(T=1 << 20, wsp=None), dict(T=1 << 20, n=4)))
    assert T.ttq_moe_sort_workspace_bytes(1 << 20, 2, 8) > 0
    for bad in ((-1, 2, 8), (4, 0, 8), (4, 2, 0), (4, 2, 2000), (1 << 30, 2, 8)):
        assert T.ttq_moe_sort_workspace_bytes(*bad) == 0


def test_gather(T):
    fn = T.lib().ttq_moe_gather
    ok = dict(X=FAKE, xt=1, T=4, K=250, ldx=256, pos=FAKE, topk=2, R=FAKE, rows=8, ldr=256, st=None)
    refuses(T, fn, ok, (dict(X=None), dict(X=FAKE + 2), dict(xt=4), dict(K=0), dict(K=257), dict(ldx=252), dict(pos=None), dict(pos=FAKE + 1), dict(topk=0),
                        dict(topk=33), dict(R=None), dict(R=FAKE + 8), dict(rows=-1), dict(ldr=248), dict(ldr=250), dict(T=-1)))
    assert fn(*dict(ok, T=0, X=None, pos=None, R=None).values()) == T.TTQ_OK
    assert fn(*dict(ok, rows=0, R=None).values()) == T.TTQ_OK


def test_combine(T):
    fn = T.lib().ttq_moe_combine
    ok = dict(R=FAKE, rt=1, rows=8, ldr=256, pos=FAKE, w=FAKE, T=4, topk=2, M=250, Y=FAKE, yt=0, ldy=251, st=None)
    refuses(T, fn, ok, (dict(R=None), dict(R=FAKE + 2), dict(rt=2), dict(rows=-1), dict(ldr=252), dict(ldr=248), dict(pos=None), dict(w=FAKE + 1),
                        dict(T=-1), dict(topk=0), dict(topk=40), dict(M=-1), dict(Y=None), dict(Y=FAKE + 2), dict(yt=2), dict(ldy=249)))
    assert fn(*dict(ok, T=0, R=None, pos=None, w=None, Y=None).values()) == T.TTQ_OK
    assert fn(*dict(ok, M=0, R=None, pos=None, w=None, Y=None).values()) == T.TTQ_OK


def test_combine_grad(T):
    fn = T.lib().ttq_moe_combine_grad
    ok = dict(dY=FAKE, yt=0, T=4, M=250, lddy=252, R=FAKE, rt=1, rows=8, ldr=256, pos=FAKE, w=FAKE, topk=2, dR=2 * FAKE, lddr=256, dw=FAKE, st=None)
    refuses(T, fn, ok, (dict(dY=None), dict(yt=2), dict(lddy=249), dict(lddy=251), dict(R=None), dict(rt=2), dict(rows=-1), dict(ldr=250), dict(pos=None),
                        dict(pos=FAKE + 2), dict(w=FAKE + 2), dict(topk=0), dict(dR=2 * FAKE + 4), dict(lddr=248), dict(lddr=252), dict(dw=FAKE + 1),
                        dict(dR=FAKE), dict(M=0), dict(T=-1)))
    assert fn(*dict(ok, T=0, dY=None, R=None, pos=None, dR=None, dw=None).values()) == T.TTQ_OK
    assert fn(*dict(ok, R=None, pos=None, dR=None, dw=None).values()) == T.TTQ_OK


def test_moe(T):
    L = T.lib()

    def call(wsp=FAKE, n=BIG, **kw):
        st = dict(s=FAKE, s_stride=0, codes=FAKE, scale=FAKE)
        gu, dn = dict(st, **kw.pop("gate_up", {})), dict(st, **kw.pop("down", {}))
        a = dict(X=FAKE, xt=1, T=4, K=256, ldx=256, ids=FAKE, w=FAKE, topk=2, E=8, I=128, M=64, gate_up=T.ExpertI8(**gu), down=T.ExpertI8(**dn), act=0,
                 Y=FAKE, yt=0, ldy=64)
        a.update(kw)
        return L.ttq_moe_i8(ctypes.byref(T.MoeI8Args(**a)), wsp, n, None)
    for bad in (dict(E=0), dict(E=1025), dict(topk=0), dict(topk=33), dict(K=250, ldx=256), dict(I=0), dict(I=100), dict(act=2), dict(xt=3), dict(yt=3),
                dict(ldx=128), dict(ldx=260), dict(ldy=63), dict(X=None), dict(X=FAKE + 8), dict(Y=None), dict(Y=FAKE + 2), dict(ids=None), dict(w=None),
                dict(ids=FAKE + 2), dict(gate_up=dict(s=None)), dict(gate_up=dict(s_stride=128)), dict(gate_up=dict(s_stride=258)),
                dict(gate_up=dict(codes=None)), dict(down=dict(codes=FAKE + 4)), dict(down=dict(scale=None)), dict(down=dict(scale=FAKE + 1)),
                dict(down=dict(s_stride=-4)), dict(M=-1), dict(T=-1), dict(wsp=None), dict(wsp=FAKE + 64), dict(n=64)):
        assert call(**bad) == T.TTQ_ERR_INVALID, bad
    for bad in (dict(K=1 << 16, ldx=1 << 16, I=1 << 15), dict(T=1 << 24), dict(T=1 << 20, K=1 << 11, ldx=1 << 11)):
        assert call(**bad) == T.TTQ_ERR_UNSUPPORTED, bad
    assert L.ttq_moe_i8(None, FAKE, BIG, None) == T.TTQ_ERR_INVALID
    assert call(T=0, X=None, ids=None, w=None, Y=None, wsp=None, n=0) == T.TTQ_OK
    assert call(M=0, Y=None, wsp=None, n=0) == T.TTQ_OK
    assert T.ttq_moe_i8_workspace_bytes(4, 2, 256, 128, 64, 8) > 0
    for bad in ((4, 0, 256, 128, 64, 8), (4, 2, 250, 128, 64, 8), (4, 2, 256, 100, 64, 8), (4, 2, 256, 128, 64, 0), (-1, 2, 256, 128, 64, 8)):
        assert T.ttq_moe_i8_workspace_bytes(*bad) == 0


def test_the_binding_takes_device_tensors_only(T):
    x = torch.zeros((2, 64))
    q, i = x.to(torch.int8), torch.zeros((2, 1), dtype=torch.int32)
    for call in (lambda: T.ttq_quantize_rows(x), lambda: T.ttq_gemm_i8(q, x[:, 0], q, x[:, 0]), lambda: T.ttq_qgemm_i8(x, None, q, x[:, 0]),
                 lambda: T.ttq_moe_sort(i, 4), lambda: T.ttq_moe_gather(x, i), lambda: T.ttq_moe_combine(x, i),
                 lambda: T.ttq_moe_combine_grad(x, x, i), lambda: T.ttq_moe_i8(x, i, i.float(), {}, {})):
        with pytest.raises(TypeError):
            call()
