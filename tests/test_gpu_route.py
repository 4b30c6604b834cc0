"""GPU parity of the router against the oracle in 64 bits: the experts exactly, the weights to 2^-20 of
them (two exponentials of 2 ulp each at most, 2^-22 together with the sum's ten roundings of 2^-24 along a
tree, a division and a product)."""
import numpy as np
import pytest
import torch

import workloads as W
from gpu_helpers import DEV, announce, need_sp
from oracle import int4_ref as R

pytestmark = pytest.mark.gpu
TOL = 2.0 ** -20


def check(logits, top, kind="softmax", bias=None, **kw):
    sp = need_sp()
    ids, w = sp.route(logits.to(DEV), top, kind=sp.ROUTE_SIGMOID if kind == "sigmoid" else sp.ROUTE_SOFTMAX,
                      bias=None if bias is None else bias.to(DEV), **kw)
    torch.cuda.synchronize()
    want, ww = R.route(logits.double().numpy(), top, sigmoid=kind == "sigmoid",
                       bias=None if bias is None else bias.double().numpy(), **kw)
    assert ids.dtype == torch.int32 and w.dtype == torch.float32
    assert np.array_equal(ids.cpu().numpy(), want)
    got = w.double().cpu().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(ww))
    ok = ~np.isnan(ww)
    assert (np.abs(got - ww)[ok] <= TOL * np.abs(ww)[ok] + 2.0 ** -149).all()


SHAPES = [(1, 1, 1, 1, 1), (1, 64, 8, 1, 1), (3, 2, 2, 1, 1), (5, 7, 3, 1, 1), (1, 60, 4, 4, 2), (300, 60, 4, 1, 1),
          (257, 128, 6, 8, 3), (130, 256, 8, 8, 4), (64, 160, 6, 8, 3), (31, 512, 10, 16, 4), (9, 1024, 64, 64, 32),
          (7, 1000, 5, 1, 1), (2, 64, 64, 1, 1), (33, 65, 2, 5, 1), (4097, 16, 2, 1, 1), (12, 100, 12, 50, 6), (6, 384, 8, 1, 1)]


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("m,e,top,groups,top_groups", SHAPES)
def test_route(m, e, top, groups, top_groups, kind, bf16):
    """Every combination of bias, group_best and renormalising; bf16 logits have many equal values."""
    l = 1.5 * torch.randn(m, e, generator=torch.Generator().manual_seed(m + e))
    l = l.to(torch.bfloat16) if bf16 else l
    bias = 0.05 * torch.randn(e, generator=torch.Generator().manual_seed(e))
    for b in (None, bias):
        for best in ((1, 2) if groups > 1 and e // groups >= 2 else (1,)):
            for renormalise in (False, True):
                announce("route", m, e, top, groups, top_groups, kind, bf16, b is not None, best, renormalise)
                check(l, top, kind, b, groups=groups, top_groups=top_groups, group_best=best, renormalise=renormalise,
                      factor=2.5 if renormalise else 1.0)


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("e,groups", [(8, 2), (64, 1), (200, 4), (256, 8), (1024, 1)])
def test_ties_go_to_the_lowest_index(kind, e, groups):
    announce("route ties", kind, e, groups)
    r = torch.Generator().manual_seed(e)
    l = torch.randint(-2, 3, (40, e), generator=r).float()
    l[0] = 1.0
    for b in (None, torch.zeros(e), torch.randint(0, 2, (e,), generator=r).float()):
        for best in (1, 2):
            check(l, min(8, e // groups), kind, b, groups=groups, top_groups=max(1, groups // 2), group_best=best)


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("e,groups", [(16, 1), (64, 4), (256, 8)])
def test_masks_and_extremes(e, groups, bf16, kind):
    """-inf masks, rows with nothing left, the types' lowest and highest values, far logits, +inf."""
    announce("route masks", e, groups, bf16, kind)
    dt = torch.bfloat16 if bf16 else torch.float32
    l = torch.randn(12, e, generator=torch.Generator().manual_seed(e)).to(dt)
    inf = float("inf")
    l[0] = -inf
    l[1, 3:] = -inf
    l[2, : e - 2] = -inf
    l[3] = torch.finfo(dt).min
    l[4, 5:] = torch.finfo(dt).min
    l[5] *= 60.0
    l[6] = -200.0 + l[6]
    l[7, 9] = inf
    l[8, 2], l[8, 7] = inf, inf
    l[9, : e // max(2, groups)] = -inf  # a whole group
    l[10] *= 1e30
    l[11] = 80.0
    top = min(4, e // groups)
    for b in (None, torch.linspace(-1.0, 1.0, e)):
        for renormalise in (False, True):
            check(l, top, kind, b, groups=groups, top_groups=max(1, groups // 2), group_best=2 if groups > 1 else 1,
                  renormalise=renormalise)


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("e", [16, 256])
def test_nan_keeps_ids_valid(e, kind):
    """A NaN is taken last; ids are different experts whatever the logits hold; other rows keep theirs."""
    sp = need_sp()
    announce("route nan", e, kind)
    l = torch.randn(6, e, generator=torch.Generator().manual_seed(1))
    k = sp.ROUTE_SIGMOID if kind == "sigmoid" else sp.ROUTE_SOFTMAX
    want = sp.route(l.to(DEV), 4, kind=k)
    l[1] = float("nan")
    l[2, 7] = float("nan")
    l[4, :-3] = float("nan")
    for b in (None, torch.zeros(e, device=DEV)):
        for groups in (1, 4):
            ids, w = sp.route(l.to(DEV), 4, kind=k, bias=b, groups=groups, top_groups=max(1, groups // 2), group_best=1)
            got = ids.cpu().numpy()
            assert all(len(set(row)) == 4 and row.min() >= 0 and row.max() < e for row in got)
            if groups == 1:
                keep = [0, 3, 5]
                assert torch.equal(ids[keep], want[0][keep])
            if groups == 1 and b is None:
                assert 7 not in got[2] and set(got[4][:3]) == {e - 3, e - 2, e - 1}


@pytest.mark.parametrize("bits", [0x7F81, 0xFF81, 0x7FC1, 0x7FFF])
def test_every_kind_of_nan(bits):
    """Signalling ones too: maxima that meet them go on to the numbers."""
    sp = need_sp()
    announce("route nan bits", hex(bits))
    for e in (16, 60, 256):
        l = torch.randn(9, e, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16)
        l.view(torch.int16)[:, 3::5] = bits - 0x10000 if bits >= 0x8000 else bits
        want, _ = R.route(l.double().numpy(), 4)
        for x in (l, l.float()):
            for b in (None, torch.zeros(e, device=DEV)):
                ids, _ = sp.route(x.to(DEV), 4, kind=sp.ROUTE_SIGMOID, bias=b)
                assert np.array_equal(ids.cpu().numpy(), want)


def test_near_scores():
    """Scores that differ by less than fp32 holds, with a bias: the order is that of 64 bits."""
    announce("route near scores")
    e = 64
    l = torch.full((50, e), 2.0)
    r = torch.Generator().manual_seed(3)
    l += torch.randint(0, 4, (50, e), generator=r).float() * 2.0 ** -21
    for kind in ("softmax", "sigmoid"):
        check(l, 6, kind, torch.full((e,), 1000.0))
        check(l, 6, kind, torch.full((e,), 0.25), groups=8, top_groups=4, group_best=2)
        check(l, 6, kind, groups=8, top_groups=4, group_best=2)


def test_given_outputs_and_graph():
    sp = need_sp()
    announce("route graph")
    l = torch.zeros(37, 256, device=DEV)
    b = torch.zeros(256, device=DEV)
    ids = torch.empty(37, 8, dtype=torch.int32, device=DEV)
    w = torch.empty(37, 8, device=DEV)
    kw = dict(kind=sp.ROUTE_SIGMOID, bias=b, groups=8, top_groups=4, group_best=2)
    assert sp.route(l, 8, ids=ids, weights=w, **kw)[0].data_ptr() == ids.data_ptr()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sp.route(l, 8, ids=ids, weights=w, **kw)
    for seed in range(3):
        l.copy_(torch.randn(37, 256, generator=torch.Generator().manual_seed(seed)))
        graph.replay()
        torch.cuda.synchronize()
        got = ids.clone(), w.clone()
        want = sp.route(l, 8, **kw)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
