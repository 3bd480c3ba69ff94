"""Host-side checks of the scored routing and 8-bit calls (no GPU needed): bad arguments come back as a status, or as
QggError from the binding, before any launch."""
import ctypes
import os

import pytest
import torch

import quantized_grouped_gemm_amd as qgg

OK, INVALID, UNSUPPORTED = 0, 1, 2
F = ctypes.c_void_p(0x1000)          # never dereferenced
ODD = ctypes.c_void_p(0x1008)        # not 16-byte aligned


@pytest.fixture
def L():
    if not os.path.exists(qgg.LIB_PATH):
        pytest.skip("libqgg.so not built")
    return qgg.lib()


def opts(score=1, n_group=1, topk_group=1, group_top=1, renorm=1, scale=1.0):
    return ctypes.byref(qgg._RouteOpts(score, n_group, topk_group, group_top, renorm, scale))


def test_route_scored(L):
    def call(T=4, E=64, k=8, typ=0, o=opts(), logits=F, ids=F):
        return L.moe_route_scored(logits, typ, None, T, E, k, o, ids, F, None, None)

    for bad in (dict(k=0), dict(k=33), dict(k=9, E=8), dict(E=1025), dict(T=-1), dict(typ=2), dict(typ=-1), dict(o=None),
                dict(logits=None), dict(ids=None), dict(o=opts(score=2)), dict(o=opts(scale=float("inf"))),
                dict(o=opts(scale=float("nan"))), dict(o=opts(n_group=0)), dict(o=opts(n_group=7)),
                dict(o=opts(n_group=8, topk_group=0)), dict(o=opts(n_group=8, topk_group=9)),
                dict(o=opts(group_top=0)), dict(o=opts(group_top=3)), dict(o=opts(n_group=64, topk_group=9, group_top=2)),
                dict(o=opts(n_group=16, topk_group=1)),            # 4 experts left for k = 8
                dict(o=opts(n_group=128), E=64)):
        assert call(**bad) == INVALID, bad
    assert call(E=1024, o=opts(n_group=128, topk_group=100)) == UNSUPPORTED
    assert call(T=0, logits=None, ids=None) == OK

    def back(T=4, E=64, k=8, typ=0, o=opts(), dl=F):
        return L.moe_route_scored_bwd(F, typ, F, F, T, E, k, o, dl, None)

    for bad in (dict(k=0), dict(k=65), dict(typ=5), dict(o=None), dict(o=opts(score=-1)), dict(dl=None)):
        assert back(**bad) == INVALID, bad
    assert back(T=0, dl=None) == OK


def test_rows(L):
    for f in (L.qgg_fp8_quantize, lambda x, m, c, a, b, s: L.qgg_fp8_dequantize(x, a, m, c, b, s)):
        assert f(F, 4, 0, F, F, None) == INVALID
        assert f(F, -1, 8, F, F, None) == INVALID
        assert f(F, 4, 12, F, F, None) == UNSUPPORTED
        assert f(F, (1 << 31) + 1, 8, F, F, None) == UNSUPPORTED
        assert f(None, 4, 8, F, F, None) == INVALID
        assert f(F, 4, 8, None, F, None) == INVALID
        assert f(F, 4, 8, F, None, None) == INVALID
        assert f(ODD, 4, 8, F, F, None) == INVALID
        assert f(None, 0, 8, None, None, None) == OK


def perm(**kw):
    p = dict.fromkeys(("counts", "offsets", "perm", "inv_perm", "active", "n_active"), 0x1000)
    p.update(kw)
    return ctypes.byref(qgg._Perm(*p.values()))


def test_grouped_gemm(L):
    def call(E=8, N=256, K=512, st=0, codes=0x1000, scales=0x1000, a=F, s=F, flags=1, p=perm(), T=4, k=2, y=F):
        w = qgg._Fp8Weight(E, N, K, st, codes, scales)
        return L.fp8_grouped_gemm(ctypes.byref(w), a, s, flags, p, T, k, y, None)

    for bad in (dict(N=0), dict(K=-128), dict(st=2), dict(codes=0), dict(scales=0), dict(codes=0x1008), dict(st=1, scales=0x1002),
                dict(a=None), dict(s=None), dict(y=None), dict(a=ODD), dict(y=ODD), dict(flags=4), dict(flags=8), dict(T=-1),
                dict(k=0), dict(k=9), dict(E=0), dict(E=1025), dict(p=None), dict(p=perm(counts=0)), dict(p=perm(perm=0)),
                dict(p=perm(inv_perm=0)), dict(p=perm(n_active=0)), dict(T=1 << 30, k=2)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(K=192), dict(N=96), dict(K=32768 + 128), dict(flags=3, N=32768 + 64), dict(N=65536, K=65536, flags=3),
                dict(N=1 << 18, K=1 << 14), dict(T=1 << 20, k=1, K=4096), dict(T=1 << 19, k=2, K=4096, flags=0)):
        assert call(**bad) == UNSUPPORTED, bad
    assert call(T=0, a=None, s=None, y=None, p=perm(perm=0, inv_perm=0)) == OK
    assert L.fp8_grouped_gemm(None, F, F, 1, perm(), 4, 2, F, None) == INVALID


def test_swiglu(L):
    def call(h=F, P=8, I=256, a=F, a8=F, s=F, h8=F, hs=F):
        return L.moe_swiglu_fp8(h, None, P, I, a, a8, s, h8, hs, None)

    for bad in (dict(P=-1), dict(I=0), dict(h=None), dict(s=None), dict(hs=None), dict(a=None, a8=None, h8=None), dict(h=ODD),
                dict(a=ODD), dict(a8=ODD), dict(h8=ODD)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(I=192), dict(P=(1 << 31) + 1)):
        assert call(**bad) == UNSUPPORTED, bad
    assert call(P=0, h=None, a=None, a8=None, h8=None) == OK

    def back(da=F, h8=F, hs=F, g=F, p=perm(), T=4, k=2, I=256, dh=F, dh8=F, ds=F, dg=F):
        return L.moe_swiglu_fp8_bwd(da, h8, hs, g, p, T, k, I, dh, dh8, ds, dg, None)

    for bad in (dict(da=None), dict(h8=None), dict(hs=None), dict(g=None), dict(p=None), dict(p=perm(inv_perm=0)), dict(T=-1),
                dict(k=0), dict(k=33), dict(I=-128), dict(ds=None), dict(dh=None, dh8=None, dg=None), dict(da=ODD), dict(dh=ODD)):
        assert back(**bad) == INVALID, bad
    assert back(I=320) == UNSUPPORTED
    assert back(T=0, da=None, dh=None, dh8=None, dg=None, p=perm(perm=0, inv_perm=0)) == OK


def test_combine(L):
    def call(rows=F, d=256, p=perm(), T=4, k=2, y=F):
        return L.moe_combine(rows, d, p, F, T, k, y, None)

    for bad in (dict(rows=None), dict(y=None), dict(d=0), dict(p=None), dict(T=-1), dict(k=0), dict(k=40), dict(rows=ODD)):
        assert call(**bad) == INVALID, bad
    assert call(d=12) == UNSUPPORTED
    assert call(T=0, rows=None, y=None, p=perm(perm=0, inv_perm=0)) == OK


def test_binding_refuses_what_the_library_cannot_see(L):
    """Types, shapes, devices and layouts, which the C calls take on trust."""
    x = torch.zeros(4, 256, dtype=torch.bfloat16)
    for call in (lambda: qgg.fp8_quantize(x),                                        # on the CPU
                 lambda: qgg.fp8_quantize(x.float()),
                 lambda: qgg.fp8_quantize(x[0]),
                 lambda: qgg.fp8_quantize([1.0]),
                 lambda: qgg.moe_route_scored(x.half(), 2),
                 lambda: qgg.moe_route_scored(x, 2),
                 lambda: qgg.moe_combine(x, None, 2, 2),
                 lambda: qgg.swiglu_fp8(x, want=("b",)),
                 lambda: qgg.Fp8Weight(x, x)):
        with pytest.raises(qgg.QggError):
            call()
    m = "meta"
    with pytest.raises(qgg.QggError, match="want a GPU"):
        qgg.moe_route_scored(torch.zeros(4, 8, device=m), 2)
    with pytest.raises(qgg.QggError, match="score"):
        qgg._route_opts("tanh", 1, 1, 1, True, 1.0)
