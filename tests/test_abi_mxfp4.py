"""Host-only checks of the MXFP4 and norm entry points: every argument is refused before any
HIP call, and workspace sizes.  Fake device addresses go only to calls that must reject them."""
import ctypes

import pytest
import torch

sp = pytest.importorskip("bf16_gemm_linear_amd", reason="libsp24.so not built")
lib = sp.lib

ENULL, ESHAPE, EALIGN, EWS, EMODE, EALIAS = -1, -2, -3, -5, -7, -8
A, B = 0x7F0000000000, 0x10000000  # fake, 16-byte aligned, far apart


def p(x):
    return ctypes.c_void_p(x)


def at(i):
    return A + i * B


def quant(x=at(0), rows=4, cols=256, c=at(1), s=at(2), f=lib.sp24_quant_mxfp4):
    return f(p(x), rows, cols, p(c), p(s), None)


def dequant(x=at(0), rows=4, cols=256, c=at(1), s=at(2)):
    return lib.sp24_dequant_mxfp4(p(c), p(s), rows, cols, p(x), None)


@pytest.mark.parametrize("f", [quant, dequant])
def test_quant_refusals(f):
    for name in ("x", "c", "s"):
        assert f(**{name: None}) == ENULL
        assert f(**{name: at(9) + 8}) == EALIGN
    for bad in (dict(rows=0), dict(cols=0), dict(cols=64), dict(cols=160), dict(rows=1 << 31), dict(cols=1 << 31),
                dict(rows=1 << 30, cols=1024)):
        assert f(**bad) == ESHAPE, bad
    assert f(c=at(0) + 16) == EALIAS
    assert f(s=at(0) + 4 * 256 * 2 - 16) == EALIAS


def test_quant_output_overlap():
    assert quant(s=at(1) + 16) == EALIAS


def gemm(m=8, n=256, k=256, x=at(0), xs=at(1), w=at(2), ws=at(3), y=at(4)):
    return lib.sp24_gemm_mxfp4(m, n, k, p(x), p(xs), p(w), p(ws), p(y), None)


def test_gemm_refusals():
    for name in ("x", "xs", "w", "ws", "y"):
        assert gemm(**{name: None}) == ENULL
        assert gemm(**{name: at(9) + 4}) == EALIGN
    for bad in (dict(m=0), dict(n=0), dict(k=0), dict(k=64), dict(k=192), dict(m=(1 << 21) + 1), dict(n=(1 << 21) + 1),
                dict(k=(1 << 24) + 128)):
        assert gemm(**bad) == ESHAPE, bad
    for name in ("x", "xs", "w", "ws"):
        assert gemm(**{name: at(4) + 16}) == EALIAS


def gated(m=8, f=256, k=256, x=at(0), xs=at(1), w=at(2), ws=at(3), h=at(4), hc=None, hs=None):
    return lib.sp24_gated_mxfp4(m, f, k, p(x), p(xs), p(w), p(ws), p(h), p(hc), p(hs), None)


def test_gated_refusals():
    for name in ("x", "xs", "w", "ws"):
        assert gated(**{name: None}) == ENULL
        assert gated(**{name: at(9) + 4}) == EALIGN
    assert gated(h=at(4) + 2) == EALIGN
    assert gated(h=None) == ENULL
    assert gated(h=None, hc=at(5)) == ENULL
    assert gated(h=None, hs=at(5)) == ENULL
    assert gated(hc=at(5)) == EMODE and gated(hs=at(5)) == EMODE
    assert gated(h=None, hc=at(5) + 4, hs=at(6)) == EALIGN
    for bad in (dict(m=0), dict(f=0), dict(k=200), dict(f=(1 << 20) + 1), dict(f=192, h=None, hc=at(5), hs=at(6))):
        assert gated(**bad) == ESHAPE, bad
    assert gated(h=at(2) + 16) == EALIAS
    assert gated(h=None, hc=at(5), hs=at(5) + 16) == EALIAS
    assert gated(h=None, hc=at(5), hs=at(1)) == EALIAS


def norm(kind=1, m=4, k=256, group=128, x=at(0), r=at(1), ro=at(2), w=at(3), eps=1e-5, o=at(4), s=at(5)):
    return lib.sp24_rmsnorm(kind, m, k, group, p(x), p(r), p(ro), p(w), eps, p(o), p(s), None)


def test_norm_refusals():
    for kind in range(5):
        for name in ("x", "w", "o") + (() if kind == 0 else ("s",)):
            assert norm(kind=kind, **{name: None}) == ENULL, (kind, name)
        for name in ("x", "r", "ro", "w", "o"):
            assert norm(kind=kind, **{name: at(9) + 8}) == EALIGN
        for bad in (dict(m=0), dict(k=0), dict(k=12), dict(k=65536 + 128), dict(m=(1 << 21) + 1)):
            assert norm(kind=kind, **bad) == ESHAPE, (kind, bad)
        for eps in (0.0, -1.0, float("nan"), float("inf")):
            assert norm(kind=kind, eps=eps) == EMODE
        assert norm(kind=kind, o=at(0)) == EALIAS
        assert norm(kind=kind, ro=at(0)) == EALIAS            # the residual may be updated in place, x not
        assert norm(kind=kind, ro=at(1) + 16) == EALIAS
    assert norm(kind=-1) == EMODE and norm(kind=5) == EMODE
    assert norm(r=None) == ENULL and norm(ro=None) == ENULL
    assert norm(s=at(9) + 2) == EALIGN
    assert norm(kind=4, s=at(9) + 8) == EALIGN
    assert norm(kind=4, k=192) == ESHAPE
    for g in (0, 4, 12, 24, 512):
        assert norm(kind=3, group=g) == ESHAPE
    assert norm(s=at(4)) == EALIAS


def ffn(m=4, d=256, f=512, x=at(0), r=at(1), ro=at(2), w=at(3), eps=1e-5, g=at(4), gs=at(5), dn=at(6), ds=at(7),
        y=at(8), wk=at(9), wkb=1 << 24):
    return lib.sp24_ffn_mxfp4(m, d, f, p(x), p(r), p(ro), p(w), eps, p(g), p(gs), p(dn), p(ds), p(y), p(wk), wkb, None)


def test_ffn_refusals():
    for name in ("x", "w", "g", "gs", "dn", "ds", "y"):
        assert ffn(**{name: None}) == ENULL, name
    for name in ("x", "r", "ro", "w", "g", "gs", "dn", "ds", "y", "wk"):
        assert ffn(**{name: at(11) + 8}) == EALIGN, name
    assert ffn(r=None) == ENULL and ffn(ro=None) == ENULL
    assert ffn(eps=0.0) == EMODE
    for bad in (dict(m=0), dict(d=200), dict(f=64), dict(d=1 << 17), dict(f=1 << 21)):
        assert ffn(**bad) == ESHAPE, bad
    need = sp.ffn_mxfp4_workspace_size(4, 256, 512)
    assert sp.ffn_mxfp4_workspace_size(0, 256, 512) == sp.ffn_mxfp4_workspace_size(4, 200, 512) == 0
    assert need > 0 and ffn(wk=None) == EWS and ffn(wkb=need - 1) == EWS
    assert ffn(y=at(0)) == EALIAS and ffn(wk=at(6)) == EALIAS and ffn(ro=at(8)) == EALIAS


def test_scale_index_is_the_storage_order():
    import numpy as np

    from oracle import mxfp4_ref as R
    for rows, cols in ((1, 128), (5, 640), (3, 1024)):
        s = torch.arange(rows * cols // 32, dtype=torch.int32).view(rows, -1).to(torch.uint8)
        stored = torch.empty(s.numel(), dtype=torch.uint8)
        stored[sp.mxfp4_scale_index(rows, cols)] = s
        assert np.array_equal(stored.numpy(), R.store_scales(s.numpy()))
    with pytest.raises(ValueError):
        sp.mxfp4_scale_index(3, 100)


def test_binding_refuses_host_tensors():
    x, w = torch.zeros(2, 128, dtype=torch.bfloat16), torch.zeros(128, dtype=torch.bfloat16)
    c, s = torch.zeros(2, 64, dtype=torch.uint8), torch.zeros(8, dtype=torch.uint8)
    for call in (lambda: sp.quant_mxfp4(x), lambda: sp.dequant_mxfp4(c, s), lambda: sp.gemm_mxfp4(c, s, c, s),
                 lambda: sp.gated_mxfp4(c, s, c, s), lambda: sp.rmsnorm(x, w), lambda: sp.ffn_mxfp4(x, w, c, s, c, s)):
        with pytest.raises(ValueError):
            call()
