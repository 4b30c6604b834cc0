"""Values of W that are 0 add nothing, on every kernel: rows and groups of zeros beside tokens with outliers, where
the quantiser's scale of such a group, 1, is hundreds of times its neighbours'; and the error of ordinary ones by
int4_bound, in which a group of zeros has no part."""
import numpy as np
import pytest
import torch

import workloads as W
from gpu_helpers import DEV, announce, need_sp
from int4_bound import bound
from oracle import int4_ref as R
from test_gpu_int4 import f64, product

pytestmark = pytest.mark.gpu


def tokens(m, k, seed):
    """N(0, 1), a channel in 50 a hundred times as large, as float64 of bf16 values."""
    x = W.randn_bf16((m, k), seed)
    x[:, 3::50] *= 100.0
    return x


def zero_weight(n, k, group, zeros, seed):
    """Rows n % 4 == 0 all zero (with a zero point of any value as their code), n % 4 == 1 zero in their first group
    alone; scales of zero groups 1, of others near 2^-9."""
    r = np.random.default_rng(seed)
    q = r.integers(0, 16, (n, k // group, group), dtype=np.uint8)
    s = R.bf16_round(np.exp2(r.uniform(-10, -8, (n, k // group))))
    z = r.integers(0, 16, s.shape, dtype=np.uint8) if zeros else np.full(s.shape, 8, np.uint8)
    empty = np.zeros(s.shape, bool)
    empty[0::4] = True
    empty[1::4, 0] = True
    q[empty], s[empty] = z[empty][:, None], 1.0
    q = q.reshape(n, k)
    t = (torch.from_numpy(R.pack(q)).to(DEV), W.bits_to_bf16(R.bits_of(s)).to(DEV),
         torch.from_numpy(z).to(DEV) if zeros else None)
    there = np.repeat(np.where(empty, 0.0, s), group, 1)  # scales of the groups that are not zero
    return t, R.dequant(q, s, z), (2 * 192 + np.abs(q - np.repeat(z.astype(float), group, 1))) * there


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("k,group", [(512, 128), (1024, 64), (544, 32), (4096, 128), (4096, 32)])
@pytest.mark.parametrize("m,n", [(1, 100), (2, 257), (3, 256), (16, 300), (40, 515), (77, 130), (300, 129), (1100, 260)])
def test_zero_rows_and_groups(m, n, k, group, zeros):
    sp = need_sp()
    announce("gemm_int4 zero groups", m, n, k, group, zeros)
    t, w, offset = zero_weight(n, k, group, zeros, m + n)
    xb = tokens(m, k, m)
    x = xb.double().numpy()
    y = f64(sp.gemm_int4(xb.to(DEV), *t))
    assert (y[:, 0::4] == 0).all()
    ref = product(x, w)
    few = product(np.abs(x), offset) if m <= 1024 else None  # beyond, (q - z) itself is multiplied
    assert (np.abs(y - ref) <= bound(ref, product(np.abs(x), np.abs(w)), k, group, few)).all()


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("tokens_", [1, 5, 29, 300, 1000])
def test_experts_of_zeros(tokens_, zeros):
    """Down weights of zeros: the block adds nothing whatever the gated products are."""
    sp = need_sp()
    d, f, group, count = 256, 384, 64, 3
    announce("experts_int4 zero weights", tokens_, zeros)
    gu = [zero_weight(2 * f, d, group, zeros, e)[0] for e in range(count)]
    r = np.random.default_rng(1)
    z = r.integers(0, 16, (count, d, f // group), dtype=np.uint8) if zeros else np.full((count, d, f // group), 8, np.uint8)
    codes = torch.from_numpy(R.pack(np.repeat(z, group, -1))).to(DEV)
    ones = torch.ones(z.shape, dtype=torch.bfloat16, device=DEV)
    ids = torch.from_numpy(np.stack([r.permutation(count)[:2] for _ in range(tokens_)]).astype(np.int32)).to(DEV)
    y = sp.experts_int4(tokens(tokens_, d, 3).to(DEV), ids, torch.ones(tokens_, 2, device=DEV), torch.stack([g[0] for g in gu]),
                        torch.stack([g[1] for g in gu]), codes, ones,
                        gu_zeros=torch.stack([g[2] for g in gu]) if zeros else None,
                        down_zeros=torch.from_numpy(z).to(DEV) if zeros else None)
    assert (y == 0).all()
