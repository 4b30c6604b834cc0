"""Every kernel and form of the integer 4-bit products, by name and with no other in its place: dense ones, and the
experts' gated and down products with last tiles of every number of rows that the kernels tell apart.

Exact cases: x of -1, 0, 1, scales a power of two times one of 1, 1.25, 1.5, 1.75 that all groups of a row share, so that sums,
and the quotients of a row's scales, are exact in fp32.  Others: int4_bound.  Experts: as test_gpu_experts."""
import numpy as np
import pytest
import torch

import workloads as W
from gpu_helpers import DEV, announce, need_sp
from int4_bound import bound
from oracle import int4_ref as R
from test_gpu_experts import experts
from test_gpu_experts_order import in_order
from test_gpu_int4 import f64, product

pytestmark = pytest.mark.gpu

SLAB = ["slab,%d,%d,%d,%d" % (mb, cbs, kp, slices) for mb in (1, 2) for cbs, kp in ((2, 4), (4, 2), (4, 3), (8, 1), (8, 2))
        for slices in (1, 3)]
TILED = ["tiled,0", "tiled,1"]


def sizes(config):
    """(tokens, n, k, group): n and tokens odd and whole, several steps and passes of K, a last step of 32 values."""
    if config == "vec":
        return [(m, n, k, g) for m in (1, 2) for n, k, g in ((1, 32, 32), (17, 96, 32), (130, 2176, 64), (1000, 4224, 128))]
    if config.startswith("slab"):
        return [(3, 1, 32, 32), (16, 130, 96, 32), (33, 515, 448, 64), (17, 64, 1152, 128), (50, 100, 2080, 32), (64, 33, 3136, 64),
                (21, 70, 10368, 128), (5, 257, 10304, 32), (300, 40, 640, 128)]
    return [(1, 1, 32, 32), (100, 300, 96, 32), (257, 513, 544, 32), (300, 130, 64, 64), (129, 257, 448, 64), (600, 260, 128, 128),
            (513, 512, 1024, 128), (20, 40, 4160, 64), (256, 256, 2048, 32)]


def put(q, s, z):
    return (torch.from_numpy(R.pack(q)).to(DEV), W.bits_to_bf16(R.bits_of(s)).to(DEV),
            None if z is None else torch.from_numpy(z).to(DEV))


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("config", ["vec"] + SLAB + TILED)
def test_named_exact(config, zeros, monkeypatch):
    sp = need_sp()
    monkeypatch.setenv("SP24_INT4", config + "!")
    for m, n, k, group in sizes(config):
        announce("exact", config, m, n, k, group, zeros)
        r = np.random.default_rng(m + n + k)
        q = r.integers(0, 16, (n, k), dtype=np.uint8)
        s = np.exp2(r.integers(-3, 2, (n, k // group))) * r.choice([-1.0, 1.0], (n, k // group)) * (1 + r.integers(0, 4, (n, 1)) / 4)
        z = r.integers(0, 256 if m % 2 else 16, s.shape, dtype=np.uint8) if zeros else None
        x = r.integers(-1, 2, (m, k)).astype(np.float64) * (r.random((m, k)) < min(1.0, 100 / k))
        # in steps of 2^-5: values below 2^5 times at most 255 + 7 / 4, and 192 + 63 times x in a kernel's sums
        assert np.abs(x).sum(1).max() * 510 * 2 ** 7 < 2 ** 24
        y = f64(sp.gemm_int4(torch.from_numpy(x).to(torch.bfloat16).to(DEV), *put(q, s, z)))
        assert np.array_equal(y, R.bf16_round(product(x, R.dequant(q, s, z)))), (m, n, k, group)


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("config", ["vec"] + SLAB + TILED)
def test_named_bound(config, zeros, monkeypatch):
    """Scales of all mantissas and both signs, a hundredth of them 0, subnormal or 1 beside a group of zeros; channels with
    outliers; the same bits on a second run."""
    sp = need_sp()
    monkeypatch.setenv("SP24_INT4", config + "!")
    for m, n, k, group in sizes(config):
        announce("bound", config, m, n, k, group, zeros)
        r = np.random.default_rng(m + n + k)
        q = r.integers(0, 16, (n, k // group, group), dtype=np.uint8)
        shape = (n, k // group)
        s = R.bf16_round(np.exp2(r.uniform(-11, -6, shape)) * r.choice([-1.0, 1.0], shape))
        z = r.integers(0, 16, shape, dtype=np.uint8) if zeros else np.full(shape, 8, np.uint8)
        odd = r.random(shape)
        s[odd < 0.01], s[odd > 0.99] = 0.0, 2.0 ** -130
        empty = (odd > 0.49) & (odd < 0.5)
        q[empty], s[empty] = z[empty][:, None], 1.0
        q = q.reshape(n, k)
        xb = W.randn_bf16((m, k), m + k)
        xb[:, :: max(1, k // 20)] *= 20.0
        x, w, dev = xb.double().numpy(), R.dequant(q, s, z), put(q, s, z if zeros else None)
        y = sp.gemm_int4(xb.to(DEV), *dev)
        few = None
        if not config.startswith("tiled"):
            there = np.repeat(np.where(empty, 0.0, np.abs(s)), group, 1)
            few = product(np.abs(x), (2 * 192 + np.abs(q - np.repeat(z.astype(float), group, 1))) * there)
        ref = product(x, w)
        assert (np.abs(f64(y) - ref) <= bound(ref, product(np.abs(x), np.abs(w)), k, group, few)).all(), (m, n, k, group)
        assert torch.equal(y, sp.gemm_int4(xb.to(DEV), *dev))


@pytest.mark.parametrize("config,m", [("vec", 2), ("slab,1,2,4,1", 40), ("slab,2,8,2,3", 40), ("tiled,0", 300), ("tiled,1", 300)])
def test_named_values_that_are_no_numbers(config, m, monkeypatch):
    """Scales of 0, NaN, Inf and the least subnormal; tokens with Inf and NaN: where they are and nowhere else."""
    sp = need_sp()
    monkeypatch.setenv("SP24_INT4", config + "!")
    for group, k in ((32, 544), (64, 448), (128, 2048)):
        announce("no numbers", config, m, k, group)
        n = 70
        r = np.random.default_rng(k)
        q = r.integers(0, 16, (n, k), dtype=np.uint8)
        s = np.exp2(r.integers(-3, 4, (n, k // group)).astype(np.float64))
        x = r.integers(-1, 2, (m, k)).astype(np.float64)
        s[3, 1], s[7, 2], s[9, 1], s[11] = 0.0, np.nan, np.inf, 2.0 ** -133
        xb = torch.from_numpy(x).to(torch.bfloat16)
        clean = np.where(np.isfinite(s), s, 1.0)
        want = R.bf16_round(product(x, R.dequant(q, clean)))
        for z in (None, np.full(s.shape, 8, np.uint8)):
            dev = put(q, s, z)
            if group == 128:  # bits_of keeps an Inf
                assert torch.isinf(dev[1].float()).sum() == 1
            y = f64(sp.gemm_int4(xb.to(DEV), *dev))
            keep = [i for i in range(n) if i not in (7, 9)]
            assert np.array_equal(y[:, keep], want[:, keep])
            assert np.isnan(y[:, 7]).all() and not np.isfinite(y[:, 9]).any()
            bad = xb.clone()
            bad[0, k - 1], bad[m - 1, 5] = float("inf"), float("nan")
            y2 = f64(sp.gemm_int4(bad.to(DEV), *dev))
            rows = [i for i in range(m) if i not in (0, m - 1)]
            assert np.array_equal(y2[rows][:, keep], y[rows][:, keep])
            assert not np.isfinite(y2[0]).any() and np.isnan(y2[m - 1]).all()


# rows of the experts: none, one, and around every boundary of the 16- and 32-row tiles and of the 64-row parts
COUNTS = [0, 1, 16, 17, 33, 64, 65, 0, 128, 129, 192, 193, 256, 257, 321]


def pairs_of(counts, seed):
    ids = np.repeat(np.arange(len(counts)), counts)
    return np.random.default_rng(seed).permutation(ids).astype(np.int32)


EXPERTS = ["slab,%d,%d,%d,1" % (mb, cbs, kp) for mb in (1, 2) for cbs, kp in ((2, 4), (4, 2), (8, 1))] + TILED


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("config", ["vec"] + EXPERTS)
@pytest.mark.parametrize("d,f,group", [(256, 384, 128), (192, 320, 64), (160, 96, 32), (2304, 128, 128), (96, 2080, 32)])
def test_named_experts(config, d, f, group, zeros, monkeypatch):
    sp = need_sp()
    monkeypatch.setenv("SP24_INT4", config + "!")
    announce("experts", config, d, f, group, zeros)
    counts = COUNTS if config != "vec" else [0, 1, 5, 9]
    args, gu, dn = experts(len(counts), d, f, group, zeros, 3, exact=True)
    one = pairs_of(counts, 1)
    tokens = len(one)
    ids = np.stack((one, np.full(tokens, -1, np.int32)), 1)  # and a slot without an expert
    ids[::2] = ids[::2, ::-1]
    r = np.random.default_rng(d)
    x = np.zeros((tokens, d))
    for t in range(tokens):
        x[t, r.choice(d, 2, replace=False)] = 1.0
    weights = np.exp2(r.integers(-2, 3, ids.shape))
    y = sp.experts_int4(torch.from_numpy(x).to(torch.bfloat16).to(DEV), torch.from_numpy(ids).to(DEV),
                        torch.from_numpy(weights).float().to(DEV), *args[:4], gu_zeros=args[4], down_zeros=args[5])
    assert np.array_equal(f64(y), R.bf16_round(in_order(x, ids, weights, gu, dn, f).astype(np.float64)))


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("config", ["vec"] + EXPERTS)
@pytest.mark.parametrize("d,f,group", [(256, 384, 128), (192, 320, 64), (544, 96, 32)])
def test_named_experts_bound(config, d, f, group, zeros, monkeypatch):
    """Random data: h's bound from the gated product's (|silu'| < 1.1, 2^-16 for the activation's arithmetic, half a bf16
    step for its rounding), carried through the down product, whose own is int4_bound's; a fp32 rounding a slot."""
    sp = need_sp()
    monkeypatch.setenv("SP24_INT4", config + "!")
    announce("experts bound", config, d, f, group, zeros)
    counts = COUNTS if config != "vec" else [0, 1, 5, 9]
    args, gu, dn = experts(len(counts), d, f, group, zeros, 5)
    one = pairs_of(counts, 2)
    ids = np.stack((one, one[::-1]), 1)
    tokens = len(one)
    xb = W.randn_bf16((tokens, d), 1)
    weights = np.random.default_rng(3).random(ids.shape).astype(np.float32)
    y = f64(sp.experts_int4(xb.to(DEV), torch.from_numpy(ids).to(DEV), torch.from_numpy(weights).to(DEV), *args[:4],
                            gu_zeros=args[4], down_zeros=args[5]))

    def err(x, part):
        _, w, q, s, z = part
        e = (x.shape[1] + 2 * s.shape[1] + 4) * 2.0 ** -23 * product(x, np.abs(w))
        if config.startswith("tiled"):
            return e
        zz = np.repeat(np.full(s.shape, 8.0) if z is None else z.astype(float), group, 1)
        return e + group * 2.0 ** -23 * product(x, (2 * 192 + np.abs(q - zz)) * np.repeat(np.abs(s), group, 1))

    x, ref, tol = xb.double().numpy(), np.zeros((tokens, d)), np.zeros((tokens, d))
    for e in range(len(counts)):
        t, slot = np.nonzero(ids == e)
        if t.size == 0:
            continue
        p, ep = product(x[t], gu[e][1]), err(np.abs(x[t]), gu[e])
        a, u, ea, eu = R.silu(p[:, :f]), p[:, f:], 1.1 * ep[:, :f], ep[:, f:]
        h = a * u
        eh = ea * np.abs(u) + np.abs(a) * eu + ea * eu
        eh += (2.0 ** -8 + 2.0 ** -16) * (np.abs(h) + eh)
        w = weights[t, slot].astype(np.float64)[:, None]
        v = product(h, dn[e][1])
        ev = err(np.abs(h) + eh, dn[e]) + product(eh, np.abs(dn[e][1]))
        np.add.at(ref, t, w * v)
        np.add.at(tol, t, w * (ev + 2.0 ** -22 * (np.abs(v) + ev)))
    assert (np.abs(y - ref) <= (2.0 ** -8 * (np.abs(ref) + tol) + tol) * (1 + 2.0 ** -20)).all()


def test_what_a_name_cannot_run(monkeypatch):
    sp = need_sp()
    announce("int4 names")
    t = put(np.full((64, 128), 9, np.uint8), np.ones((64, 1)), None)
    x = torch.ones(3, 128, dtype=torch.bfloat16, device=DEV)
    for name in ("vec!", "slab,3,2,4,1!", "slab,1,4,8,1!", "slab,1,2!", "tiled,2!", "other!"):
        monkeypatch.setenv("SP24_INT4", name)
        with pytest.raises(sp.Sp24Error):
            sp.gemm_int4(x, *t)
    for name in ("vec", "slab,3,2,4,1", "tiled,2", "other"):  # the planner's own
        monkeypatch.setenv("SP24_INT4", name)
        assert (sp.gemm_int4(x, *t) == 128).all()
