"""int4_bound is tight enough to tell: exact products summed in fp32 stay inside it, and what a kernel might do instead does
not (planted here on the host)."""
import numpy as np
import pytest

import workloads as W
from int4_bound import bound
from oracle import int4_ref as R


def data(k, group, seed=0):
    r = np.random.default_rng(seed)
    q = r.integers(0, 16, (40, k), dtype=np.uint8)
    s = R.bf16_round(np.exp2(r.uniform(-11, -6, (40, k // group))) * r.choice([-1.0, 1.0], (40, k // group)))
    x = W.randn_bf16((30, k), k).double().numpy()
    x[:, :: max(1, k // 20)] *= 20.0
    return x, q, s, R.dequant(q, s)


def inside(y, x, w, k, group):
    ref = x @ w.T
    return (np.abs(R.bf16_round(y) - ref) <= bound(ref, np.abs(x) @ np.abs(w).T, k, group)).all()


@pytest.mark.parametrize("k,group", [(448, 64), (544, 32), (1024, 128)])
def test_bound(k, group):
    x, q, s, w = data(k, group)
    v = (q.astype(np.float64) - 8).astype(np.float32)
    acc = np.zeros((30, 40), np.float32)
    for g in range(k // group):
        part = np.zeros((30, 40), np.float32)
        for i in range(g * group, (g + 1) * group):
            part += x[:, i].astype(np.float32)[:, None] * v[:, i][None]
        acc += part * s[:, g].astype(np.float32)
    assert inside(acc.astype(np.float64), x, w, k, group)
    # values of W rounded to bf16, scales cut to six bits, one group's scale a bf16 step off, one code off by one
    assert not inside(x @ R.bf16_round(w).T, x, w, k, group)
    e = np.exp2(np.floor(np.log2(np.abs(s))))
    assert not inside(x @ R.dequant(q, np.sign(s) * np.floor(np.abs(s) / e * 64) / 64 * e).T, x, w, k, group)
    off = s.copy()
    off[:, 1] *= 1 + 2.0 ** -7
    assert not inside(x @ R.dequant(q, off).T, x, w, k, group)
    code = q.copy()
    code[:, 7] ^= 1
    assert not inside(x @ R.dequant(code, s).T, x, w, k, group)
