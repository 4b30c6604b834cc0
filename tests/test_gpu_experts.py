"""GPU parity of the experts' block over integer 4-bit weights against 64 bits.

Exact cases: tokens of a few ones, gates of at least 32 (where silu(g) is g in fp32), powers of two for
scales and weights: h and y are exact, so y is the bf16 rounding.  Others: the product's bound (see
test_gpu_int4) carried through h = silu(g) u (|silu'| < 1.1), 2^-8 |h| for its rounding to bf16 and 2^-16
for the activation's own arithmetic, then through the down product, and 2^-8 |y|."""
import numpy as np
import pytest
import torch

import workloads as W
from gpu_helpers import DEV, announce, need_sp
from oracle import int4_ref as R
from test_gpu_int4 import f64, product, weight

pytestmark = pytest.mark.gpu


def stack(parts):
    return [None if p[0] is None else torch.stack(p) for p in zip(*parts)]


def experts(count, d, f, group, zeros, seed, exact=False):
    """(arguments of the call, per expert the float64 gate-up and down values and their parts)."""
    gu = [weight(2 * f, d, group, zeros, seed + 2 * e, exact) for e in range(count)]
    dn = [weight(d, f, group, zeros, seed + 2 * e + 1, exact) for e in range(count)]
    if exact:  # gates 32 to 224, ups and down weights of at most 15 in magnitude
        r = np.random.default_rng(seed)

        def again(part, gates):
            _, _, q, s, z = part
            q, s = q.copy(), r.choice([-1.0, 1.0], s.shape)
            if gates:
                q[:f], s[:f] = 9 + q[:f] % 7, 32.0
                z = None if z is None else np.full_like(z, 8)
            return ((torch.from_numpy(R.pack(q)).to(DEV), W.bits_to_bf16(R.bits_of(s)).to(DEV),
                     None if z is None else torch.from_numpy(z).to(DEV)), R.dequant(q, s, z), q, s, z)

        gu, dn = [again(p, True) for p in gu], [again(p, False) for p in dn]
    gt, dt = stack([w[0] for w in gu]), stack([w[0] for w in dn])
    return (gt[0], gt[1], dt[0], dt[1], gt[2], dt[2]), gu, dn


def error(x, part, extra=None):
    """Bound of a product's error; extra: the operand's own error."""
    _, w, q, s, z = part
    group, k = q.shape[1] // s.shape[1], q.shape[1]
    zz = np.full(s.shape, 8.0) if z is None else z
    big = (128 + np.maximum(q, np.repeat(zz, group, 1))) * np.repeat(np.abs(s), group, 1)
    e = 2.0 ** -16 * product(np.abs(x), big) + (k / 32 + 16) * 2.0 ** -24 * product(np.abs(x), np.abs(w))
    return e if extra is None else e + product(extra, np.abs(w))


def reference(x, ids, weights, gu, dn, f):
    """(y, bound) in float64."""
    y, tol = np.zeros((x.shape[0], dn[0][1].shape[0])), np.zeros((x.shape[0], dn[0][1].shape[0]))
    for e in range(len(gu)):
        token, slot = np.nonzero(ids == e)
        if token.size == 0:
            continue
        p, ep = product(x[token], gu[e][1]), error(x[token], gu[e])
        g, u, eg, eu = p[:, :f], p[:, f:], ep[:, :f], ep[:, f:]
        a = R.silu(g)
        h = a * u
        eh = 1.1 * eg * np.abs(u) + np.abs(a) * eu + 1.1 * eg * eu
        eh = eh + (2.0 ** -8 + 2.0 ** -16) * (np.abs(h) + eh)
        w = weights[token, slot][:, None]
        np.add.at(y, token, w * product(h, dn[e][1]))
        np.add.at(tol, token, np.abs(w) * error(np.abs(h) + eh, dn[e], eh))
    return y, tol * (1 + 2.0 ** -20) + 2.0 ** -8 * np.abs(y)


def choose(tokens, count, top, seed, skew=False):
    r = np.random.default_rng(seed)
    like = r.random((tokens, count)) + (3.0 * (np.arange(count) < 2) if skew else 0.0)
    return np.argsort(-like, 1)[:, :top].astype(np.int32)


SHAPES = [(1, 2, 1, 32, 32, 32), (1, 64, 8, 512, 256, 128), (3, 8, 2, 128, 96, 32), (8, 4, 4, 256, 128, 64), (29, 16, 8, 384, 640, 128),
          (70, 5, 3, 192, 64, 64), (130, 3, 2, 1024, 256, 128), (257, 32, 4, 256, 512, 64), (700, 8, 2, 256, 384, 128),
          (33, 128, 1, 64, 64, 32), (16, 1, 1, 416, 224, 32), (1000, 4, 4, 128, 128, 128), (2, 1024, 64, 32, 32, 32),
          (1100, 2, 2, 512, 1088, 64), (4, 6, 2, 4096, 1792, 128), (1, 8, 8, 4096, 1792, 128)]


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("tokens,count,top,d,f,group", SHAPES)
def test_exact(tokens, count, top, d, f, group, zeros):
    sp = need_sp()
    announce("experts_int4 exact", tokens, count, top, d, f, group, zeros)
    args, gu, dn = experts(count, d, f, group, zeros, 7 * tokens, exact=True)
    r = np.random.default_rng(tokens)
    x = np.zeros((tokens, d))
    for t in range(tokens):
        x[t, r.choice(d, 2, replace=False)] = 1.0
    ids = choose(tokens, count, top, tokens, skew=True)
    weights = np.exp2(r.integers(-2, 1, ids.shape))
    y = sp.experts_int4(torch.from_numpy(x).to(torch.bfloat16).to(DEV), torch.from_numpy(ids).to(DEV),
                        torch.from_numpy(weights).float().to(DEV), *args[:4], gu_zeros=args[4], down_zeros=args[5])
    torch.cuda.synchronize()
    # h is 32 times an integer of at most 8 bits; sums of h (q - z) in steps of 32, of weighted ones in steps of 8
    want, size = np.zeros((tokens, d)), np.zeros((tokens, d))
    for e in range(count):
        token, slot = np.nonzero(ids == e)
        if token.size:
            p = product(x[token], gu[e][1])
            h = p[:, :f] * p[:, f:]
            assert np.array_equal(h, R.bf16_round(h)) and np.abs(h).max() * 143 * 128 / 32 < 2 ** 24
            np.add.at(want, token, weights[token, slot][:, None] * product(h, dn[e][1]))
            np.add.at(size, token, weights[token, slot][:, None] * product(np.abs(h), np.abs(dn[e][1])))
    assert size.max() / 8 < 2 ** 24
    assert np.array_equal(f64(y), R.bf16_round(want))


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("tokens,count,top,d,f,group", SHAPES)
def test_experts(tokens, count, top, d, f, group, zeros):
    sp = need_sp()
    announce("experts_int4", tokens, count, top, d, f, group, zeros)
    args, gu, dn = experts(count, d, f, group, zeros, tokens)
    xb = W.randn_bf16((tokens, d), tokens)
    ids = choose(tokens, count, top, tokens + 1, skew=tokens % 2 == 1)
    weights = np.random.default_rng(3).random(ids.shape).astype(np.float32)
    call = lambda: sp.experts_int4(xb.to(DEV), torch.from_numpy(ids).to(DEV), torch.from_numpy(weights).to(DEV),
                                   *args[:4], gu_zeros=args[4], down_zeros=args[5])
    y = call()
    torch.cuda.synchronize()
    ref, tol = reference(xb.double().numpy(), ids, weights.astype(np.float64), gu, dn, f)
    assert (np.abs(f64(y) - ref) <= tol).all()
    assert torch.equal(y, call())


@pytest.mark.parametrize("tokens", [1, 5, 40, 600])
def test_ids_outside_and_twice(tokens):
    """Pairs without an expert add nothing, a token without any is 0, an expert twice adds twice; the
    other tokens keep their bits."""
    sp = need_sp()
    announce("experts_int4 ids", tokens)
    count, top, d, f = 6, 3, 256, 128
    args, gu, dn = experts(count, d, f, 64, True, 5)
    xb = W.randn_bf16((tokens, d), 2)
    ids = choose(tokens, count, top, 4)
    weights = np.random.default_rng(3).random(ids.shape).astype(np.float32)

    def call(i):
        return sp.experts_int4(xb.to(DEV), torch.from_numpy(i).to(DEV), torch.from_numpy(weights).to(DEV), *args[:4],
                               gu_zeros=args[4], down_zeros=args[5])

    before = call(ids)
    other = ids.copy()
    other[0] = [-1, count, 1 << 30]
    if tokens > 1:
        other[1, 0] = -(1 << 31)
        other[2] = other[2, 0]
    y = call(other)
    torch.cuda.synchronize()
    ref, tol = reference(xb.double().numpy(), other, weights.astype(np.float64), gu, dn, f)
    assert (np.abs(f64(y) - ref) <= tol).all() and (y[0] == 0).all()
    if tokens < 5:
        return
    # the other tokens: only their rows' places moved
    ref, tol = reference(xb.double().numpy(), ids, weights.astype(np.float64), gu, dn, f)
    assert (np.abs(f64(before) - ref) <= tol).all()
    assert torch.equal(y[3:], before[3:])


def test_everything_to_one_expert():
    sp = need_sp()
    announce("experts_int4 one expert")
    count, d, f = 40, 128, 160
    args, gu, dn = experts(count, d, f, 32, False, 9)
    for tokens in (1, 20, 333):
        xb = W.randn_bf16((tokens, d), tokens)
        ids = np.full((tokens, 1), 37, np.int32)
        w = np.ones((tokens, 1), np.float32)
        y = sp.experts_int4(xb.to(DEV), torch.from_numpy(ids).to(DEV), torch.from_numpy(w).to(DEV), *args[:4])
        torch.cuda.synchronize()
        ref, tol = reference(xb.double().numpy(), ids, w.astype(np.float64), gu, dn, f)
        assert (np.abs(f64(y) - ref) <= tol).all()


def test_nan_token_stays_in_its_row():
    sp = need_sp()
    announce("experts_int4 nan")
    count, top, d, f = 4, 2, 128, 64
    args, *_ = experts(count, d, f, 64, False, 11)
    for tokens in (6, 90, 700):
        x = W.randn_bf16((tokens, d), 1).to(DEV)
        ids = torch.from_numpy(choose(tokens, count, top, 8)).to(DEV)
        w = torch.full((tokens, top), 0.5, device=DEV)
        want = sp.experts_int4(x, ids, w, *args[:4])
        x[2, 3] = float("nan")
        y = sp.experts_int4(x, ids, w, *args[:4])
        torch.cuda.synchronize()
        keep = [i for i in range(tokens) if i != 2]
        assert torch.isnan(y[2]).all() and torch.equal(y[keep], want[keep])


def test_workspaces_and_graph():
    """Two captured calls with workspaces of their own, replayed with eager calls between."""
    sp = need_sp()
    announce("experts_int4 graph")
    count, top, d, f = 8, 2, 256, 128
    args, *_ = experts(count, d, f, 128, False, 13)
    for tokens in (1, 24, 300):
        x = torch.zeros(tokens, d, dtype=torch.bfloat16, device=DEV)
        ids = torch.zeros(tokens, top, dtype=torch.int32, device=DEV)
        w = torch.full((tokens, top), 0.5, device=DEV)
        outs = [torch.empty_like(x), torch.empty_like(x)]
        ws = [torch.empty(sp.experts_int4_workspace_size(tokens, d, f, count, top), dtype=torch.uint8, device=DEV)
              for _ in outs]

        def run():
            sp.experts_int4(x, ids, w, *args[:4], out=outs[0], ws=ws[0])
            sp.experts_int4(outs[0], ids, w, *args[:4], out=outs[1], ws=ws[1])

        run()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            run()
        for seed in range(3):
            x.copy_(W.randn_bf16((tokens, d), seed))
            ids.copy_(torch.from_numpy(choose(tokens, count, top, seed)))
            graph.replay()
            torch.cuda.synchronize()
            got = [o.clone() for o in outs]
            first = sp.experts_int4(x, ids, w, *args[:4])
            assert torch.equal(got[0], first) and torch.equal(got[1], sp.experts_int4(first, ids, w, *args[:4]))
