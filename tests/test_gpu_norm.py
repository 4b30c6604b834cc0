"""GPU parity of sp24_rmsnorm against the oracle in 64 bits.

The kernel's v is t rstd w in fp32: rstd carries the error of a sum of at most 65536 squares (a
tree of at most 64 + 10 + 16 adds in a row: 90 roundings of 2^-24, halved by the square root) and
five more roundings, so |v - v64| <= 2^-18 |v64|; scales and codes follow from that."""
import numpy as np
import pytest
import torch

import workloads as W
from gpu_helpers import DEV, announce, bits, codes, need_sp
from oracle import mxfp4_ref as R
from oracle import sp24_ref as O
from test_gpu_mxfp4 import check_mx4_output, np8

pytestmark = pytest.mark.gpu
REL = 2.0 ** -18


def inputs(m, k, seed, residual):
    x = W.randn_bf16((m, k), seed).float()
    x[:, :: max(2, k // 3)] *= 30.0
    if m > 2:
        x[m // 2] *= 1e4
    r = W.randn_bf16((m, k), seed + 1).float() if residual else None
    if m > 3:
        x[m - 1] = 0.0
        if residual:
            r[m - 1] = 0.0
    w = (1 + 0.2 * W.randn_bf16((k,), seed + 2).float()).to(torch.bfloat16)
    bf = lambda t: None if t is None else t.to(torch.bfloat16)
    return bf(x), bf(r), w


def run(kind, m, k, group, residual, seed):
    sp = need_sp()
    announce("rmsnorm kind", kind, m, k, group, residual)
    x, r, w = inputs(m, k, seed, residual)
    o, s, ro = sp.rmsnorm(x.to(DEV), w.to(DEV), kind, residual=None if r is None else r.to(DEV), eps=1e-5, group=group)
    torch.cuda.synchronize()
    v, t = R.norm_ref(W.bf16_bits(x), None if r is None else W.bf16_bits(r), W.bf16_bits(w), 1e-5)
    if residual:  # the fp32 sum rounded once: one of the two neighbours at an fp32 tie
        got = O.bf16_to_f64(bits(ro))
        assert (np.abs(got - t) <= 2.0 ** -8 * np.abs(t) * (1 + 2.0 ** -14)).all()
        t32 = W.bf16_bits((x.float() + r.float()).to(torch.bfloat16))
        assert np.array_equal(bits(ro), t32)
    else:
        assert ro is None
    return o, s, v


# lengths at the edges of the threads-per-row choices, and odd ones
LENGTHS = [8, 24, 128, 512, 520, 1000, 2048, 2056, 4096, 4104, 8192, 8200, 14336, 16384, 16392, 65536]


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("k", LENGTHS)
def test_bf16(k, residual):
    sp = need_sp()
    for m in (1, 2, 7):
        o, s, v = run(sp.NORM_BF16, m, k, 0, residual, k + m)
        assert s is None
        assert (np.abs(O.bf16_to_f64(bits(o)) - v) <= (2.0 ** -8 + REL) * np.abs(v)).all()


def check_codes(q, s, v, top, integer):
    """s = amax / top and q within half a step of v / s, v and s each within REL."""
    amax = np.abs(v).max(-1, keepdims=True)
    s64 = np.where(amax > 0, amax / top, 1.0)
    assert (np.abs(s - s64[..., 0]) <= 2 * REL * s64[..., 0]).all()
    a = v / s64
    if integer:
        step = 1.0
    else:
        step = 2.0 ** (np.maximum(np.floor(np.log2(np.maximum(np.abs(a), 2.0 ** -20))), -6) - 3)
    assert (np.abs(q - np.clip(a, -top, top)) <= 0.5 * step + 4 * REL * np.abs(a)).all()
    assert (np.abs(q) <= top).all()


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("k", LENGTHS)
def test_rows_fp8_and_int8(k, residual):
    sp = need_sp()
    for m in (1, 5):
        o, s, v = run(sp.NORM_FP8_ROWS, m, k, 0, residual, k + m)
        check_codes(O.e4m3_decode(codes(o)).astype(np.float64), s.cpu().numpy().astype(np.float64), v,
                    448.0, False)
        o, s, v = run(sp.NORM_INT8_ROWS, m, k, 0, residual, k + m)
        check_codes(o.cpu().numpy().astype(np.float64), s.cpu().numpy().astype(np.float64), v, 127.0, True)


@pytest.mark.parametrize("k,group", [(8, 8), (128, 32), (384, 24), (640, 128), (1536, 384), (2048, 2048), (4096, 128),
                                     (4096, 512), (4608, 4608), (8192, 1024), (14336, 256), (16384, 8), (65520, 24)])
def test_groups(k, group):
    sp = need_sp()
    for m, residual in ((1, True), (6, False), (9, True)):
        o, s, v = run(sp.NORM_FP8_GROUPS, m, k, group, residual, k + group + m)
        q = o.view(torch.float8_e4m3fn).float().cpu().double().numpy()
        g = k // group
        check_codes(q.reshape(m * g, group), s.cpu().numpy().astype(np.float64).reshape(-1), v.reshape(m * g, group),
                    448.0, False)


@pytest.mark.parametrize("k", [128, 640, 1920, 4096, 8192, 14336, 65536])
def test_mxfp4(k):
    sp = need_sp()
    for m, residual in ((1, True), (4, False), (7, True)):
        o, s, v = run(sp.NORM_MXFP4, m, k, 0, residual, k + m)
        check_mx4_output(o, s, v, REL * np.abs(v), (m, k))


# above 2^21 values short rows take several vectors a thread (below, one: the tests above), whose
# rows and groups end inside a thread's vectors; a part of the rows is compared
@pytest.mark.parametrize("m,k,group", [(2101, 1000, 200), (2049, 1024, 128), (1281, 1664, 104), (1050, 2048, 8),
                                       (1031, 2040, 408), (1000, 2176, 128), (523, 4096, 512), (600, 3648, 24)])
def test_short_rows_in_number(m, k, group):
    sp = need_sp()
    assert m * k > 1 << 21
    x, r, w = inputs(m, k, m + k, True)
    xd, rd, wd = x.to(DEV), r.to(DEV), w.to(DEV)
    pick = np.r_[0:3, m // 2 - 2 : m // 2 + 3, m - 4 : m]
    v, t = R.norm_ref(W.bf16_bits(x[pick]), W.bf16_bits(r[pick]), W.bf16_bits(w), 1e-5)
    for kind in (sp.NORM_BF16, sp.NORM_FP8_ROWS, sp.NORM_INT8_ROWS, sp.NORM_FP8_GROUPS, sp.NORM_MXFP4):
        if kind == sp.NORM_MXFP4 and k % 128:
            continue
        announce("rmsnorm kind", kind, m, k, group)
        o, s, ro = sp.rmsnorm(xd, wd, kind, residual=rd, eps=1e-5, group=group)
        torch.cuda.synchronize()
        assert np.array_equal(bits(ro), W.bf16_bits((x.float() + r.float()).to(torch.bfloat16)))
        if kind == sp.NORM_BF16:
            assert (np.abs(O.bf16_to_f64(bits(o)[pick]) - v) <= (2.0 ** -8 + REL) * np.abs(v)).all()
        elif kind == sp.NORM_MXFP4:
            part = torch.from_numpy(R.store_scales(R.load_scales(np8(s), m, k)[pick]))
            check_mx4_output(o[torch.from_numpy(pick).to(DEV)], part, v, REL * np.abs(v), (m, k))
        else:
            q = o.float() if kind == sp.NORM_INT8_ROWS else o.view(torch.float8_e4m3fn).float()
            q, s = q.cpu().double().numpy()[pick], s.cpu().numpy().astype(np.float64)[pick]
            g = k // group if kind == sp.NORM_FP8_GROUPS else 1
            check_codes(q.reshape(-1, k // g), s.reshape(-1), v.reshape(-1, k // g),
                        127.0 if kind == sp.NORM_INT8_ROWS else 448.0, kind == sp.NORM_INT8_ROWS)


def test_residual_in_place_and_many_rows():
    sp = need_sp()
    for m, k in ((4099, 128), (1031, 4096)):
        announce("rmsnorm in place", m, k)
        x, r, w = (t.to(DEV) for t in inputs(m, k, m, True))
        o, s, ro = sp.rmsnorm(x, w, sp.NORM_FP8_ROWS, residual=r)
        r2 = r.clone()
        o2, s2, ro2 = sp.rmsnorm(x, w, sp.NORM_FP8_ROWS, residual=r2, residual_out=r2)
        torch.cuda.synchronize()
        assert ro2 is r2
        assert torch.equal(ro.view(torch.int16), r2.view(torch.int16))
        assert torch.equal(o, o2) and torch.equal(s, s2)


def test_zero_tiny_huge_and_nonfinite_rows():
    sp = need_sp()
    announce("rmsnorm special rows")
    k = 1024
    x = torch.randn(8, k, generator=torch.Generator().manual_seed(0))
    x[1] = 0.0
    x[2] *= 1e-38
    x[3] *= 1e15
    x[4, 77] = float("inf")
    x[5, 78] = float("nan")
    x[6, 1:] = 0.0
    x = x.to(torch.bfloat16)
    w = torch.ones(k, dtype=torch.bfloat16)
    v, _ = R.norm_ref(W.bf16_bits(x), None, W.bf16_bits(w), 1e-6)
    fin = [0, 1, 2, 3, 6, 7]
    xd, wd = x.to(DEV), w.to(DEV)
    for kind, top in ((sp.NORM_FP8_ROWS, 448.0), (sp.NORM_INT8_ROWS, 127.0)):
        o, s, _ = sp.rmsnorm(xd, wd, kind)
        torch.cuda.synchronize()
        q = (o.float() if kind == sp.NORM_INT8_ROWS else o.view(torch.float8_e4m3fn).float()).cpu().double().numpy()
        s = s.cpu().numpy().astype(np.float64)
        check_codes(q[fin], s[fin], v[fin], top, kind == sp.NORM_INT8_ROWS)
        assert s[1] == 1.0 and not q[1].any()
        assert np.isnan(s[[4, 5]]).all() and not q[[4, 5]].any()
    o, s, _ = sp.rmsnorm(xd, wd, sp.NORM_MXFP4)
    torch.cuda.synchronize()
    b = R.load_scales(np8(s), 8, k)
    assert (b[1] == 127).all() and (b[5] == 255).all() and b[4, 77 // 32] == 255
    rows = torch.tensor(fin, device=DEV)
    sf = torch.from_numpy(R.store_scales(b[fin])).to(DEV)
    check_mx4_output(o[rows], sf, v[fin], REL * np.abs(v[fin]), "special")


def test_feeds_the_sparse_products():
    """The 8-bit forms go straight into the sparse products of the library."""
    sp = need_sp()
    m, n, k = 7, 300, 1024
    announce("rmsnorm into gemm_rows and gemm_groups")
    x, r, w = inputs(m, k, 5, True)
    v, _ = R.norm_ref(W.bf16_bits(x), W.bf16_bits(r), W.bf16_bits(w), 1e-6)
    wv, meta = sp.prune_compress(W.randn_bf16((n, k), 6, 0.02).to(DEV))
    args = x.to(DEV), w.to(DEV)
    dense = O.bf16_to_f64(bits(sp.decompress(wv, meta, k)))
    ref = v @ dense.T
    # E4M3 steps are 2^-4 of a value at most, INT8's 1/254 of the row's largest, on both sides
    for kind, quant in ((sp.NORM_FP8_ROWS, sp.quant_fp8), (sp.NORM_INT8_ROWS, sp.quant_int8)):
        q, s, _ = sp.rmsnorm(*args, kind, residual=r.to(DEV))
        wq, sw = quant(wv)
        y = sp.gemm_rows(q, wq, meta, s, sw)
        torch.cuda.synchronize()
        err = np.linalg.norm(O.bf16_to_f64(bits(y)) - ref) / np.linalg.norm(ref)
        assert err < 0.15, err
    q, s, _ = sp.rmsnorm(*args, sp.NORM_FP8_GROUPS, residual=r.to(DEV), group=128)
    gq, gs = sp.quant_fp8_groups(wv, 64)
    y = sp.gemm_groups(q, s, gq, meta, gs, group=128)
    torch.cuda.synchronize()
    err = np.linalg.norm(O.bf16_to_f64(bits(y)) - ref) / np.linalg.norm(ref)
    assert err < 0.15, err
