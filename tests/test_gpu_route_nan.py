"""GPU parity of the router on logits with NaN: such an expert is masked as one of -inf is, it comes last with
weight 0, and the others' scores, choices and weights are those of a row without it.

Weights: formed in 64 bits and rounded once to fp32, so 2^-24 of them (and half the least subnormal); 2^-20 of
that again for the oracle's own exponentials."""
import numpy as np
import pytest
import torch

from gpu_helpers import DEV, announce, need_sp
from oracle import int4_ref as R

pytestmark = pytest.mark.gpu


def check(l, masked, top, kind, bias, **kw):
    """l's ids and weights are the oracle's of `masked`, the same with -inf in place of NaN."""
    sp = need_sp()
    ids, w = sp.route(l.to(DEV), top, kind=sp.ROUTE_SIGMOID if kind == "sigmoid" else sp.ROUTE_SOFTMAX,
                      bias=None if bias is None else bias.to(DEV), **kw)
    torch.cuda.synchronize()
    want, ww = R.route(masked.double().numpy(), top, sigmoid=kind == "sigmoid",
                       bias=None if bias is None else bias.double().numpy(), **kw)
    assert np.array_equal(ids.cpu().numpy(), want)
    assert (np.abs(w.double().cpu().numpy() - ww) <= 2.0 ** -24 * (1 + 2.0 ** -20) * ww + 2.0 ** -150).all()


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("e,groups", [(5, 1), (16, 4), (60, 1), (64, 8), (256, 8), (512, 1), (1000, 1), (1024, 4)])
def test_nan_is_masked(e, groups, kind, bf16):
    l = 1.5 * torch.randn(10, e, generator=torch.Generator().manual_seed(e))
    r = np.random.default_rng(e)
    where = torch.zeros(10, e, dtype=torch.bool)
    where[1, 0] = True                                      # the first
    where[2, int(l[2].argmax())] = True                     # what would be the best
    where[3] = True                                         # all
    where[4, 2:] = True                                     # fewer numbers than are chosen
    where[5] = torch.from_numpy(r.random(e) < 0.5)
    where[6, : e // max(2, groups)] = True                  # a whole group
    where[7, 1] = True
    l[7, 2] = float("inf")
    where[8, ::2] = True                                    # beside masks of -inf
    l[8, 1::4] = float("-inf")
    l = l.to(torch.bfloat16) if bf16 else l
    masked = l.clone()
    masked[where] = float("-inf")
    l[where] = float("nan")
    top = min(4, e // groups)
    for b in (None, torch.zeros(e), 0.05 * torch.randn(e, generator=torch.Generator().manual_seed(1))):
        for best in ((1, 2) if groups > 1 else (1,)):
            for renormalise in (False, True):
                announce("route nan", e, groups, kind, bf16, b is not None, best, renormalise)
                check(l, masked, top, kind, b, groups=groups, top_groups=max(1, groups // 2), group_best=best,
                      renormalise=renormalise, factor=1.5)


@pytest.mark.parametrize("bits", [0x7F81, 0xFF81, 0x7FC1, 0xFFFF])
def test_every_kind_of_nan_has_weight_0(bits):
    announce("route nan bits", hex(bits))
    for e in (16, 256):
        l = torch.randn(9, e, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16)
        masked = l.clone()
        masked[:, 3:] = float("-inf")
        l.view(torch.int16)[:, 3:] = bits - 0x10000 if bits >= 0x8000 else bits
        for kind in ("softmax", "sigmoid"):
            for b in (None, torch.zeros(e)):
                for renormalise in (False, True):
                    check(l, masked, 5, kind, b, renormalise=renormalise)
                    check(l.float(), masked, 5, kind, b, renormalise=renormalise)


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
def test_weights_are_rounded_once(kind):
    """No NaN: the same bound on ordinary rows."""
    announce("route weights", kind)
    for m, e in ((300, 60), (100, 256), (50, 1024)):
        l = 3.0 * torch.randn(m, e, generator=torch.Generator().manual_seed(m))
        for b in (None, 0.05 * torch.randn(e, generator=torch.Generator().manual_seed(e))):
            for renormalise in (False, True):
                check(l, l, 6, kind, b, renormalise=renormalise)
