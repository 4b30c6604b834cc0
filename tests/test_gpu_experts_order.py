"""The experts' sum over a token's slots, for calls of every size alike: each slot's product finished, times its weight, in
fp32 in the order of the slots.

The products are exact (see test_gpu_experts), the weights powers of two, so the sums can be followed in fp32 on the
host; a token's first and last slots are one expert with weights 2^26 and -2^26, so that what the others lose
beside them stays in the result."""
import numpy as np
import pytest
import torch

import workloads as W
from gpu_helpers import DEV, announce, need_sp
from oracle import int4_ref as R
from test_gpu_experts import experts
from test_gpu_int4 import f64, product

pytestmark = pytest.mark.gpu


def in_order(x, ids, weights, gu, dn, f):
    """fp32 [tokens, d], slot after slot."""
    y = np.zeros((x.shape[0], dn[0][1].shape[0]), np.float32)
    for j in range(ids.shape[1]):
        v = np.zeros(y.shape)
        for e in np.unique(ids[:, j]):
            t = np.flatnonzero(ids[:, j] == e)
            if 0 <= e < len(gu):
                p = product(x[t], gu[e][1])
                h = p[:, :f] * p[:, f:]
                assert np.array_equal(h, R.bf16_round(h))
                v[t] = product(h, dn[e][1])
        assert np.array_equal(v, v.astype(np.float32))
        y = (y.astype(np.float64) + weights[:, j, None] * v).astype(np.float32)  # the product is exact
    return y


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("tokens,count,top,d,f,group", [(1, 12, 10, 64, 64, 32), (4, 12, 12, 96, 96, 32), (1, 3, 2, 128, 4224, 128),
                                                        (2, 5, 3, 64, 2112, 64), (1, 64, 64, 32, 32, 32), (1, 4, 9, 128, 4352, 128),
                                                        (40, 12, 10, 64, 64, 32), (500, 12, 9, 128, 128, 64)])
def test_order(tokens, count, top, d, f, group, zeros):
    sp = need_sp()
    announce("experts_int4 order", tokens, count, top, d, f, group, zeros)
    args, gu, dn = experts(count, d, f, group, zeros, 3, exact=True)
    r = np.random.default_rng(tokens + top)
    x = np.zeros((tokens, d))
    for t in range(tokens):
        x[t, r.choice(d, 2, replace=False)] = 1.0
    ids = r.integers(0, count, (tokens, top)).astype(np.int32)
    ids[r.random(ids.shape) < 0.1] = -1
    ids[:, -1] = ids[:, 0] = r.integers(0, count, tokens)
    weights = np.exp2(r.integers(0, 3, ids.shape)) * r.choice([-1.0, 1.0], ids.shape)
    weights[:, 0], weights[:, -1] = 2.0 ** 26, -(2.0 ** 26)
    y = sp.experts_int4(torch.from_numpy(x).to(torch.bfloat16).to(DEV), torch.from_numpy(ids).to(DEV),
                        torch.from_numpy(weights).float().to(DEV), *args[:4], gu_zeros=args[4], down_zeros=args[5])
    assert np.array_equal(f64(y), R.bf16_round(in_order(x, ids, weights, gu, dn, f).astype(np.float64)))


@pytest.mark.parametrize("tokens", [1, 3, 64, 700])
@pytest.mark.parametrize("small", [False, True])
def test_weights_far_from_the_scales(tokens, small):
    """A weight times a scale that leaves fp32's range, where the result is well inside."""
    sp = need_sp()
    announce("experts_int4 weights", tokens, small)
    count, top, d, f, group = 4, 2, 64, 64, 32
    sign = -1 if small else 1
    gu_scale = np.ones((count, 2 * f, d // group))
    gu_scale[:, f:] = 2.0 ** (-75 * sign)
    q = np.full((count, 2 * f, d), 8, np.uint8)
    q[:, :f, 0], q[:, f:, 0] = 12, 9              # x = 16: gates 64, ups 16 of their scale
    dq = np.random.default_rng(1).integers(0, 16, (count, d, f), dtype=np.uint8)
    dn_scale = np.full((count, d, f // group), 2.0 ** (60 * sign))

    def put(v, s):
        return torch.from_numpy(R.pack(v)).to(DEV), W.bits_to_bf16(R.bits_of(s)).to(DEV)

    x = torch.zeros(tokens, d)
    x[:, 0] = 16.0
    ids = torch.from_numpy(np.stack([np.random.default_rng(t).permutation(count)[:top] for t in range(tokens)]).astype(np.int32))
    w = 2.0 ** (90 * sign)
    y = sp.experts_int4(x.to(torch.bfloat16).to(DEV), ids.to(DEV), torch.full((tokens, top), w, device=DEV),
                        *put(q, gu_scale), *put(dq, dn_scale))
    h = 64.0 * 16.0 * 2.0 ** (-75 * sign)
    per = np.stack([h * (v.astype(np.float64) - 8).sum(1) * 2.0 ** (60 * sign) for v in dq])  # exact in fp32
    want = (w * per[ids.numpy()]).sum(1)
    assert np.array_equal(f64(y), R.bf16_round(want))
