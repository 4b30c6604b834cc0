"""sp24_rmsnorm where t w leaves fp32's range and v = t w / sqrt(mean t^2 + eps) does not.

Values are held to the oracle in 64 bits by the bounds of test_gpu_norm: v carries at most 2^-18
(its rows' sums are of the same length), and scales and codes follow from it; a bf16 value also half
of its type's least subnormal, 2^-134."""
import numpy as np
import pytest
import torch

import workloads as W
from gpu_helpers import DEV, announce, bits, codes, need_sp
from oracle import mxfp4_ref as R
from oracle import sp24_ref as O
from test_gpu_mxfp4 import check_mx4_output
from test_gpu_norm import REL, check_codes

pytestmark = pytest.mark.gpu

# the rows' size and the weight's: products of 1e42, 1e40, 1e-40, 1e-44 and 1e-46
SIZES = [(1e12, 1e30), (1e4, 1e36), (1e-20, 1e-20), (1e-14, 1e-30), (1e-13, 1e-33)]
# one to eight vectors a thread, and one, two and four rows a workgroup
SHAPES = [(5, 512), (9, 1024), (3, 4096), (3, 8192), (2, 40960)]


def by_kind(sp, kind, o, s, v, group):
    m, k = v.shape
    if kind == sp.NORM_BF16:
        assert (np.abs(O.bf16_to_f64(bits(o)) - v) <= (2.0 ** -8 + REL) * np.abs(v) + 2.0 ** -134).all()
    elif kind == sp.NORM_MXFP4:
        check_mx4_output(o, s, v, REL * np.abs(v), (m, k))
    else:
        per = group if kind == sp.NORM_FP8_GROUPS else k
        q = o.cpu().numpy() if kind == sp.NORM_INT8_ROWS else O.e4m3_decode(codes(o))
        check_codes(q.astype(np.float64).reshape(-1, per), s.cpu().numpy().astype(np.float64).reshape(-1),
                    v.reshape(-1, per), 127.0 if kind == sp.NORM_INT8_ROWS else 448.0, kind == sp.NORM_INT8_ROWS)


@pytest.mark.parametrize("size,weight", SIZES)
def test_large_and_small_weights(size, weight):
    """Groups of 128 and 512 lie in a wave, groups of 1024 in several."""
    sp = need_sp()
    eps = 1e-37
    for m, k in SHAPES:
        x = (W.randn_bf16((m, k), m + k).float() * size).to(torch.bfloat16)
        w = ((1 + 0.2 * W.randn_bf16((k,), k).float()) * weight).to(torch.bfloat16)
        v, _ = R.norm_ref(W.bf16_bits(x), None, W.bf16_bits(w), eps)
        assert np.isfinite(v).all()
        for kind in range(5):
            for group in ((128, 1024 if k % 1024 == 0 else 512) if kind == sp.NORM_FP8_GROUPS else (128,)):
                announce("rmsnorm range", kind, m, k, group, size, weight)
                o, s, _ = sp.rmsnorm(x.to(DEV), w.to(DEV), kind, eps=eps, group=group)
                torch.cuda.synchronize()
                by_kind(sp, kind, o, s, v, group)


@pytest.mark.parametrize("k", [384, 768, 2048, 4608])
def test_one_row_out_of_range_among_others(k):
    """Rows in range keep their bits beside rows that are not, whatever shares a workgroup with them:
    four, two and one row each; groups of 64 lie in a wave, those of half a row in LDS."""
    sp = need_sp()
    w = ((1 + 0.2 * W.randn_bf16((k,), k).float()) * 1e30).to(torch.bfloat16)
    x = W.randn_bf16((7, k), 3).float()
    x[[1, 6]] *= 1e12
    x[4] = 0.0
    x = x.to(torch.bfloat16)
    r = (W.randn_bf16((7, k), 4).float() * (x.float().abs().amax(-1, keepdim=True) > 0)).to(torch.bfloat16)
    v, _ = R.norm_ref(W.bf16_bits(x), W.bf16_bits(r), W.bf16_bits(w), 1e-5)
    for kind in range(5):
        for group in ((64, k // 2) if kind == sp.NORM_FP8_GROUPS else (128,)):
            announce("rmsnorm mixed rows", kind, k, group)
            o, s, ro = sp.rmsnorm(x.to(DEV), w.to(DEV), kind, residual=r.to(DEV), eps=1e-5, group=group)
            torch.cuda.synchronize()
            by_kind(sp, kind, o, s, v, group)
            for i in range(7):
                o1, s1, ro1 = sp.rmsnorm(x[i:i + 1].to(DEV), w.to(DEV), kind, residual=r[i:i + 1].to(DEV), eps=1e-5,
                                         group=group)
                torch.cuda.synchronize()
                assert torch.equal(o1.view(torch.uint8)[0], o.view(torch.uint8)[i])
                assert torch.equal(ro1.view(torch.int16)[0], ro.view(torch.int16)[i])
                if kind not in (sp.NORM_BF16, sp.NORM_MXFP4):
                    assert torch.equal(s1.view(torch.int32)[0], s.view(torch.int32)[i])


def test_one_group_out_of_range():
    """A group whose products fall below fp32's range beside others of its row that do not; groups of
    one wave's lanes, of parts of several waves, and not a power of two."""
    sp = need_sp()
    for k, group in ((2048, 128), (4096, 1024), (4608, 1536), (3840, 240)):
        x = W.randn_bf16((3, k), k).float()
        w = 1 + 0.2 * W.randn_bf16((k,), k + 1).float()
        x[:, group:2 * group] *= 1e-10
        w[group:2 * group] *= 1e-24
        x, w = (x * 1e-12).to(torch.bfloat16), w.to(torch.bfloat16)
        v, _ = R.norm_ref(W.bf16_bits(x), None, W.bf16_bits(w), 1e-30)
        announce("rmsnorm one group", k, group)
        o, s, _ = sp.rmsnorm(x.to(DEV), w.to(DEV), sp.NORM_FP8_GROUPS, eps=1e-30, group=group)
        torch.cuda.synchronize()
        by_kind(sp, sp.NORM_FP8_GROUPS, o, s, v, group)


@pytest.mark.parametrize("k,group", [(512, 64), (384, 192), (2048, 128), (8192, 1024), (4608, 1536), (40960, 512)])
def test_groups_of_zeros(k, group):
    """A group of zeros (of x, of the weight, of one lane's values) gets scale 1 and codes 0, the row's other
    groups what they get without it: their codes do not depend on the sum of squares."""
    sp = need_sp()
    x, w = W.randn_bf16((4, k), k).float(), 1 + 0.2 * W.randn_bf16((k,), 3).float()
    x[1, group:2 * group] = 0.0
    x[2, group:group + 8] = 0.0
    x[3] = 0.0
    x = x.to(torch.bfloat16)
    for zero in (False, True):
        if zero:
            w[:group] = 0.0
        wb = w.to(torch.bfloat16)
        v, _ = R.norm_ref(W.bf16_bits(x), None, W.bf16_bits(wb), 1e-5)
        announce("rmsnorm zeros", k, group, zero)
        o, s, _ = sp.rmsnorm(x.to(DEV), wb.to(DEV), sp.NORM_FP8_GROUPS, eps=1e-5, group=group)
        torch.cuda.synchronize()
        by_kind(sp, sp.NORM_FP8_GROUPS, o, s, v, group)
        assert (s[1, 1] == 1).item() and (s[3] == 1).all().item() and not o.view(torch.uint8)[1, group:2 * group].any().item()
        y = x.clone()
        y[1, group:2 * group] = 1.0
        o2, _, _ = sp.rmsnorm(y.to(DEV), wb.to(DEV), sp.NORM_FP8_GROUPS, eps=1e-5, group=group)
        torch.cuda.synchronize()
        assert torch.equal(o.view(torch.uint8)[1, 2 * group:], o2.view(torch.uint8)[1, 2 * group:])
