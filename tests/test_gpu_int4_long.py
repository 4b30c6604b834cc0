"""Experts whose weights lie beyond 4 GiB from the first, and X rows beyond it: offsets past 32 bits."""
import numpy as np
import pytest
import torch

import workloads as W
from gpu_helpers import DEV, announce, need_sp
from test_gpu_experts import experts, reference
from test_gpu_int4 import f64

pytestmark = pytest.mark.gpu


def test_weights_beyond_4_gib():
    sp = need_sp()
    count, d, f, group = 700, 4096, 1792, 128  # gate-up codes: 5.1 GB
    announce("experts_int4 far weights")
    args, gu, dn = experts(1, d, f, group, False, 21)
    far = [torch.zeros((count, *t.shape[1:]), dtype=t.dtype, device=DEV) for t in args[:4]]
    assert far[0].numel() > 1 << 32
    for a, t in zip(far, args[:4]):
        a[-1] = t[0]
    for tokens in (1, 30, 90):
        xb = W.randn_bf16((tokens, d), tokens)
        ids = torch.full((tokens, 1), count - 1, dtype=torch.int32, device=DEV)
        w = torch.ones((tokens, 1), device=DEV)
        y = sp.experts_int4(xb.to(DEV), ids, w, *far)
        torch.cuda.synchronize()
        ref, tol = reference(xb.double().numpy(), np.zeros((tokens, 1), np.int32), np.ones((tokens, 1)), gu, dn, f)
        assert (np.abs(f64(y) - ref) <= tol).all(), tokens


def test_tokens_beyond_4_gib():
    """The last tokens of a call whose X is larger than 4 GiB, at sizes that the tiled kernel takes."""
    sp = need_sp()
    tokens, d, f, count = 280000, 8192, 32, 2
    announce("experts_int4 far tokens")
    args, gu, dn = experts(count, d, f, 32, True, 23)
    x = torch.zeros((tokens, d), dtype=torch.bfloat16, device=DEV)
    assert x.numel() * 2 > 1 << 32
    xb = W.randn_bf16((5, d), 3)
    x[-5:] = xb.to(DEV)
    ids = torch.zeros((tokens, 1), dtype=torch.int32, device=DEV)
    ids[1::2] = 1
    w = torch.ones((tokens, 1), device=DEV)
    y = sp.experts_int4(x, ids, w, *args[:4], gu_zeros=args[4], down_zeros=args[5])
    torch.cuda.synchronize()
    ref, tol = reference(xb.double().numpy(), ids[-5:].cpu().numpy(), np.ones((5, 1)), gu, dn, f)
    assert (np.abs(f64(y[-5:]) - ref) <= tol).all()
    assert not y[:-5].any()
