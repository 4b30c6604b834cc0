"""GPU parity of the integer 4-bit quantiser and product against the oracle in 64 bits.

Codes, scales and zero points bit for bit.  Products of small integers with scales that are powers of
two are exact in fp32 in any order, so they must be the bf16 rounding of the exact sum.  Of other data:
|y - ref| <= 2^-8 |ref| + 2^-17 A + (k / 32 + 16) 2^-24 B.  The first term is half a bf16 step.  A = sum of |x|
(128 + max(q, z)) |s|, twice over: a kernel may form x (128 + q) and x (128 + z) apart; a group's sum has at most
128 / 32 + 32 roundings or truncations of 2^-23, below 2^-17.8.  B = sum |x w|, joined over at most k / 32 groups
and 16 waves in fp32.  Where a kernel multiplies (q - z) and rescales its sums a group at a time, it rounds them
3 k / 32 times (an instruction every 16 values, a quotient and a product a group) by 2^-24 of at most B, and
A >= 8 B."""
import numpy as np
import pytest
import torch

import workloads as W
from gpu_helpers import DEV, announce, bits, need_sp
from oracle import int4_ref as R

pytestmark = pytest.mark.gpu


def weight(n, k, group, zeros, seed, exact=False):
    """Random codes, scales and zero points: (tensors on the GPU, values float64, q, s, z)."""
    r = np.random.default_rng(seed)
    q = r.integers(0, 16, (n, k), dtype=np.uint8)
    s = np.exp2(r.integers(-3, 4, (n, k // group))) if exact else R.bf16_round(
        np.exp2(r.uniform(-9, -6, (n, k // group))) * r.choice([-1.0, 1.0], (n, k // group), p=[0.1, 0.9]))
    z = r.integers(0, 16, (n, k // group), dtype=np.uint8) if zeros else None
    t = (torch.from_numpy(R.pack(q)).to(DEV), W.bits_to_bf16(R.bits_of(s)).to(DEV),
         None if z is None else torch.from_numpy(z).to(DEV))
    return t, R.dequant(q, s, z), q, s, z


def product(x, w):
    """x w^T in float64 on the GPU."""
    return (torch.from_numpy(x).to(DEV) @ torch.from_numpy(w).to(DEV).t()).cpu().numpy()


def tolerance(x, w, q, s, z, ref):
    group, k = q.shape[1] // s.shape[1], q.shape[1]
    zz = np.full(s.shape, 8.0) if z is None else z
    big = (128 + np.maximum(q, np.repeat(zz, group, 1))) * np.repeat(np.abs(s), group, 1)
    return (2.0 ** -8 * np.abs(ref) + 2.0 ** -16 * product(np.abs(x), big) +
            (k / 32 + 16) * 2.0 ** -24 * product(np.abs(x), np.abs(w)))


def f64(y):
    return y.double().cpu().numpy()


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("rows,cols,group", [(1, 32, 32), (1, 128, 128), (3, 192, 64), (17, 4096, 128), (1000, 96, 32),
                                             (64, 14336, 64), (70001, 128, 32), (9001, 2176, 128)])
def test_quant_bit_exact(rows, cols, group, zeros):
    sp = need_sp()
    announce("quant_int4", rows, cols, group, zeros)
    x = W.randn_bf16((rows, cols), rows + cols).float()
    x[0, ::7] *= 1000.0
    x[-1, :group] = 0.0
    x[0, 0] += 3.0
    xb = x.to(torch.bfloat16)
    q, s, z = R.quant(W.bf16_bits(xb), group, zeros)
    c, sc, zp = sp.quant_int4(xb.to(DEV), group=group, zeros=zeros)
    v = sp.dequant_int4(c, sc, zp)
    torch.cuda.synchronize()
    assert np.array_equal(bits(sc), R.bits_of(s))
    assert np.array_equal(c.cpu().numpy(), R.pack(q))
    assert zp is None if z is None else np.array_equal(zp.cpu().numpy(), z)
    assert np.array_equal(f64(v), R.bf16_round(R.dequant(q, s, z)))
    assert torch.equal(sp.unpack_int4(c).cpu(), torch.from_numpy(q))
    assert torch.equal(sp.pack_int4(sp.unpack_int4(c)), c)


@pytest.mark.parametrize("zeros", [False, True])
def test_quant_extremes(zeros):
    """Subnormals, the largest values (their range is beyond fp32), infinities, NaN, ties."""
    sp = need_sp()
    announce("quant_int4 extremes", zeros)
    b = np.zeros((12, 64), np.uint16)
    r = np.random.default_rng(5)
    b[0] = r.integers(0, 1 << 16, 64)                       # any patterns
    b[1, :32] = r.integers(1, 128, 32)                      # subnormals
    b[2, 3] = 1                                             # one, the least: its scale is 1
    b[3, 0], b[3, 1] = 0x7F7F, 0xFF7F                       # +-max
    b[4, 9], b[5, 40], b[6, 1] = 0x7F80, 0xFF80, 0x7FC1     # Inf, -Inf, NaN
    b[7] = 0x8000                                           # -0
    b[8] = W.bf16_bits((torch.arange(64) * 0.5 - 16).to(torch.bfloat16))  # ties
    b[9:] = r.integers(0, 0x7F80, (3, 64)) | (r.integers(0, 2, (3, 64)) << 15)
    q, s, z = R.quant(b, 32, zeros)
    c, sc, zp = sp.quant_int4(W.bits_to_bf16(b).to(DEV), group=32, zeros=zeros)
    torch.cuda.synchronize()
    assert np.array_equal(bits(sc), R.bits_of(s))
    assert np.array_equal(c.cpu().numpy(), R.pack(q))
    assert z is None or np.array_equal(zp.cpu().numpy(), z)


SHAPES = [(1, 1, 32, 32), (1, 16, 128, 128), (1, 14336, 4096, 128), (2, 17, 96, 32), (3, 100, 4096, 64), (8, 4096, 14336, 128),
          (16, 515, 1088, 64), (17, 256, 1152, 128), (33, 1000, 2080, 32), (64, 384, 4096, 32), (77, 6144, 4096, 32),
          (65, 33, 128, 128), (129, 640, 448, 64), (256, 512, 2048, 128), (300, 1001, 544, 32), (1000, 129, 256, 128),
          (513, 2049, 1024, 64), (2047, 768, 8192, 128), (5, 3, 131072, 128), (200, 70, 16384, 32), (1, 70001, 64, 64),
          (4500, 40, 96, 32)]


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("m,n,k,group", SHAPES)
def test_product_exact(m, n, k, group, zeros):
    """Integers whose sums stay below 2^24 with any order and any offset of the codes."""
    sp = need_sp()
    announce("gemm_int4 exact", m, n, k, group, zeros)
    r = np.random.default_rng(m + n + k)
    t, w, q, s, z = weight(n, k, group, zeros, n * k, exact=True)
    x = r.integers(-1, 2, (m, k)).astype(np.float64) * (r.random((m, k)) < min(1.0, 256 / k))
    # a group's sum: at most 128 * 143; over the row, in steps of 2^-3, about 256 values of at most 15 * 8
    assert np.abs(x).sum(1).max() * 15 * 8 * 8 < 2 ** 24
    y = sp.gemm_int4(torch.from_numpy(x).to(torch.bfloat16).to(DEV), *t)
    torch.cuda.synchronize()
    assert np.array_equal(f64(y), R.bf16_round(product(x, w)))


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("m,n,k,group", SHAPES)
def test_product(m, n, k, group, zeros):
    sp = need_sp()
    announce("gemm_int4", m, n, k, group, zeros)
    t, w, q, s, z = weight(n, k, group, zeros, n + k)
    xb = W.randn_bf16((m, k), m + k)
    xb[:, :: max(1, k // 20)] *= 20.0
    x = xb.double().numpy()
    out = torch.full((m, n), float("nan"), dtype=torch.bfloat16, device=DEV)
    y = sp.gemm_int4(xb.to(DEV), *t, out=out)
    torch.cuda.synchronize()
    assert y.data_ptr() == out.data_ptr()
    ref = product(x, w)
    assert (np.abs(f64(y) - ref) <= tolerance(x, w, q, s, z, ref)).all()
    assert torch.equal(y, sp.gemm_int4(xb.to(DEV), *t))  # the same bits again


@pytest.mark.parametrize("m", [1, 9, 40, 200, 700])
def test_any_zero_byte(m):
    """Zero points are bytes: up to 255, not only the quantiser's 0..15."""
    sp = need_sp()
    announce("gemm_int4 zero bytes", m)
    n, k, group = 200, 256, 32
    t, _, q, s, _ = weight(n, k, group, True, 8, exact=True)
    z = np.random.default_rng(9).integers(0, 256, s.shape, dtype=np.uint8)
    x = np.random.default_rng(m).integers(-1, 2, (m, k)).astype(np.float64)
    y = sp.gemm_int4(torch.from_numpy(x).to(torch.bfloat16).to(DEV), t[0], t[1], torch.from_numpy(z).to(DEV))
    torch.cuda.synchronize()
    assert np.array_equal(f64(y), R.bf16_round(product(x, R.dequant(q, s, z))))


@pytest.mark.parametrize("m", [3, 20, 70, 300, 1100])
def test_rows_are_their_own(m):
    """An Inf or a NaN in a token stays in its row; the other rows keep their bits."""
    sp = need_sp()
    announce("gemm_int4 non-finite rows", m)
    n, k = 272, 512
    t, *_ = weight(n, k, 64, True, 4)
    x = W.randn_bf16((m, k), m).to(DEV)
    want = sp.gemm_int4(x, *t)
    x[1, 5], x[m - 1, k - 1] = float("inf"), float("nan")
    y = sp.gemm_int4(x, *t)
    torch.cuda.synchronize()
    keep = [i for i in range(m) if i not in (1, m - 1)]
    assert torch.equal(y[keep], want[keep])
    assert not torch.isfinite(y[1]).any() and torch.isnan(y[m - 1]).all()


def test_scales_zero_and_nan():
    """A group with scale 0 adds nothing, one with scale NaN makes its column NaN."""
    sp = need_sp()
    announce("gemm_int4 scales")
    t, w, q, s, z = weight(48, 256, 32, False, 6, exact=True)
    s[3, 2], s[7, 1] = 0.0, np.nan
    sc = W.bits_to_bf16(R.bits_of(s)).to(DEV)
    for m in (1, 30, 500):
        x = np.random.default_rng(m).integers(-1, 2, (m, 256)).astype(np.float64)
        y = f64(sp.gemm_int4(torch.from_numpy(x).to(torch.bfloat16).to(DEV), t[0], sc))
        assert np.isnan(y[:, 7]).all()
        keep = [i for i in range(48) if i != 7]
        assert np.array_equal(y[:, keep], R.bf16_round(product(x, R.dequant(q[keep], s[keep]))))


def test_other_stream_and_graph():
    """On a stream of the caller's, and from a graph replayed on new tokens between eager calls."""
    sp = need_sp()
    announce("gemm_int4 stream and graph")
    ws = [weight(n, 1024, 128, True, n)[0] for n in (96, 2000)]
    for m in (1, 30, 400):
        x = torch.zeros(m, 1024, dtype=torch.bfloat16, device=DEV)
        outs = [torch.empty(m, w[0].shape[0], dtype=torch.bfloat16, device=DEV) for w in ws]
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            for w, o in zip(ws, outs):
                sp.gemm_int4(x, *w, out=o)
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            for w, o in zip(ws, outs):
                sp.gemm_int4(x, *w, out=o)
        for seed in range(3):
            x.copy_(W.randn_bf16((m, 1024), seed))
            graph.replay()
            torch.cuda.synchronize()
            got = [o.clone() for o in outs]
            for w, g in zip(ws, got):
                assert torch.equal(g, sp.gemm_int4(x, *w))
