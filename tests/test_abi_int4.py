"""Host-only checks of the integer 4-bit, router and experts entry points: every argument is refused
before any HIP call, and workspace sizes.  Fake device addresses go only to calls that must reject them."""
import ctypes

import pytest
import torch

sp = pytest.importorskip("bf16_gemm_linear_amd", reason="libsp24.so not built")
lib = sp.lib

ENULL, ESHAPE, EALIGN, EDTYPE, EWS, EMODE, EALIAS = -1, -2, -3, -4, -5, -7, -8
A, B = 0x7F0000000000, 0x10000000  # fake, 16-byte aligned, far apart


def p(x):
    return ctypes.c_void_p(x)


def at(i):
    return A + i * B


def quant(w=at(0), rows=4, cols=256, group=64, c=at(1), s=at(2), z=at(3)):
    return lib.sp24_quant_int4(p(w), rows, cols, group, p(c), p(s), p(z), None)


def dequant(w=at(0), rows=4, cols=256, group=64, c=at(1), s=at(2), z=at(3)):
    return lib.sp24_dequant_int4(p(c), p(s), p(z), rows, cols, group, p(w), None)


@pytest.mark.parametrize("f", [quant, dequant])
def test_quant_refusals(f):
    for name in ("w", "c", "s"):
        assert f(**{name: None}) == ENULL
    for name in ("w", "c", "s", "z"):
        assert f(**{name: at(9) + 8}) == EALIGN
    for bad in (dict(rows=0), dict(cols=0), dict(cols=32), dict(cols=96), dict(group=0), dict(group=16), dict(group=96),
                dict(group=256), dict(group=-64), dict(rows=(1 << 21) + 1), dict(cols=(1 << 20) + 64)):
        assert f(**bad) == ESHAPE, bad
    assert f(c=at(0) + 16) == EALIAS
    assert f(s=at(0) + 4 * 256 * 2 - 16) == EALIAS
    assert f(z=at(0) + 16) == EALIAS


def test_quant_output_overlap():
    assert quant(s=at(1) + 16) == EALIAS
    assert quant(z=at(1) + 496) == EALIAS
    assert quant(z=at(2) + 16) == EALIAS


def gemm(m=8, n=256, k=4096, group=128, x=at(0), c=at(1), s=at(2), z=at(3), y=at(4), ws=at(5), ws_bytes=1 << 27):
    return lib.sp24_gemm_int4(m, n, k, group, p(x), p(c), p(s), p(z), p(y), p(ws), ws_bytes, None)


def test_gemm_refusals():
    for name in ("x", "c", "s", "y"):
        assert gemm(**{name: None}) == ENULL
    need = sp.gemm_int4_workspace_size(8, 256, 4096)
    assert need > 0 and gemm(ws=None) == EWS and gemm(ws_bytes=need - 1) == EWS
    assert sp.gemm_int4_workspace_size(1, 256, 4096) == 0 and sp.gemm_int4_workspace_size(0, 256, 4096) == 0
    assert sp.gemm_int4_workspace_size(8, 256, 100) == 0
    for name in ("x", "c", "s", "z", "y", "ws"):
        assert gemm(**{name: at(9) + 4}) == EALIGN
    for bad in (dict(m=0), dict(n=0), dict(k=0), dict(k=192), dict(k=64), dict(group=48), dict(m=(1 << 21) + 1),
                dict(n=(1 << 21) + 1), dict(k=(1 << 20) + 128), dict(m=-1)):
        assert gemm(**bad) == ESHAPE, bad
    for name in ("x", "c", "s", "z"):
        assert gemm(**{name: at(4) + 8 * 256 * 2 - 16}) == EALIAS, name
        assert gemm(**{name: at(5) + need - 16}) == EALIAS, name
    assert gemm(y=at(5)) == EALIAS


def router(kind=0, fp32=1, experts=64, top=8, groups=1, top_groups=1, best=1, renormalise=1, factor=1.0, tokens=4,
           l=at(0), b=at(1), i=at(2), w=at(3), r=True):
    st = sp._RouterStruct(kind, fp32, experts, top, groups, top_groups, best, renormalise, factor)
    return lib.sp24_route(ctypes.byref(st) if r else None, tokens, p(l), p(b), p(i), p(w), None)


def test_route_refusals():
    for name in ("l", "i", "w"):
        assert router(**{name: None}) == ENULL
    assert router(r=False) == ENULL
    for name in ("l", "b", "i", "w"):
        assert router(**{name: at(9) + 4}) == EALIGN
    assert router(kind=2) == EMODE and router(kind=-1) == EMODE
    assert router(fp32=2) == EDTYPE
    assert router(best=0) == EMODE and router(best=3) == EMODE
    assert router(factor=float("nan")) == EMODE and router(factor=float("inf")) == EMODE
    for bad in (dict(tokens=0), dict(tokens=(1 << 21) + 1), dict(experts=0), dict(experts=1025), dict(top=0), dict(top=65),
                dict(groups=0), dict(groups=5), dict(groups=8, top_groups=9), dict(groups=8, top_groups=0),
                dict(groups=16, top_groups=1, top=5), dict(groups=64, top_groups=64, best=2),
                dict(experts=256, groups=128), dict(experts=4)):
        assert router(**bad) == ESHAPE, bad
    assert router(i=at(0) + 16) == EALIAS and router(w=at(1) + 16) == EALIAS and router(w=at(2) + 16) == EALIAS


def experts(count=4, d=128, f=64, group=32, tokens=4, top=2, gc=at(0), gs=at(1), gz=at(2), dc=at(3), ds=at(4), dz=at(5),
            x=at(6), i=at(7), w=at(8), y=at(9), ws=at(10), ws_bytes=1 << 30, e=True):
    st = sp._ExpertsStruct(count, d, f, group, gc, gs, gz, dc, ds, dz)
    return lib.sp24_experts_int4(ctypes.byref(st) if e else None, tokens, top, p(x), p(i), p(w), p(y), p(ws), ws_bytes,
                                 None)


def test_experts_refusals():
    for name in ("gc", "gs", "dc", "ds", "x", "i", "w", "y"):
        assert experts(**{name: None}) == ENULL
    assert experts(e=False) == ENULL
    for name in ("gc", "gs", "gz", "dc", "ds", "dz", "x", "i", "w", "y", "ws"):
        assert experts(**{name: at(12) + 4}) == EALIGN, name
    for bad in (dict(count=0), dict(count=1025), dict(d=0), dict(d=96, group=64), dict(f=48), dict(f=96, group=64),
                dict(group=16), dict(tokens=0), dict(top=0), dict(top=65), dict(tokens=1 << 20, top=3),
                dict(d=(1 << 20) + 32)):
        assert experts(**bad) == ESHAPE, bad
    need = sp.experts_int4_workspace_size(4, 128, 64, 4, 2)
    assert need > 0
    assert experts(ws=None) == EWS and experts(ws_bytes=need - 1) == EWS
    for name in ("gc", "gs", "gz", "dc", "ds", "dz", "x", "i", "w"):
        assert experts(**{name: at(9) + 16}) == EALIAS, name
        assert experts(**{name: at(10) + need - 16}) == EALIAS, name
    assert experts(y=at(10) + 256) == EALIAS


def test_workspace_sizes():
    size = sp.experts_int4_workspace_size
    assert size(0, 128, 64, 4, 2) == 0 and size(4, 100, 64, 4, 2) == 0 and size(4, 128, 64, 0, 2) == 0
    assert size(1 << 20, 32, 32, 4, 3) == 0
    # the pairs' order, h in bf16 and outputs in fp32 fit
    assert size(100, 128, 64, 4, 2) >= 4 * 5 + 200 * (4 + 2 * 64 + 4 * 128)


def test_pack_refusals():
    for bad in (torch.zeros(2, 12, dtype=torch.uint8), torch.zeros(2, 16, dtype=torch.int32),
                torch.zeros((), dtype=torch.uint8)):
        with pytest.raises(ValueError):
            sp.pack_int4(bad)
    with pytest.raises(ValueError):
        sp.unpack_int4(torch.zeros(2, 6, dtype=torch.uint8))


def test_binding_wants_gpu_tensors():
    w, c, s = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(4, 2)
    i = torch.zeros(4, 1, dtype=torch.int32)
    for call in (lambda: sp.quant_int4(w), lambda: sp.dequant_int4(c, s), lambda: sp.gemm_int4(w, c, s),
                 lambda: sp.route(s, 1), lambda: sp.experts_int4(w, i, s, c, s, c, s)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: sp.quant_int4(), lambda: sp.route(s), lambda: sp.gemm_int4(w, c), lambda: sp.route(s, 1, grups=2),
                 lambda: sp.quant_int4("w")):
        with pytest.raises(TypeError):
            call()
