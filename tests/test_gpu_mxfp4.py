"""GPU parity of the MXFP4 operators against the NumPy oracle in 64 bits.

Codes and scales of the quantiser are compared bit for bit.  Products: |y - ref| <= 2^-8 |ref| +
2^-15 sum|x w|; the first term is half a bf16 ulp, the second fp32 accumulation (at most k/64 + 64
roundings or truncations of a partial sum of at most sum|x w|, each 2^-23: below 2^-15 up to
k = 16384).  The gated product carries that error through h = silu(g) u (|silu'| < 1.1), plus 2^-16
|h| for the activation's own arithmetic."""
import numpy as np
import pytest
import torch

import workloads as W
from gpu_helpers import DEV, announce, bits, need_sp
from oracle import mxfp4_ref as R
from oracle.sp24_ref import bf16_to_f64

pytestmark = pytest.mark.gpu
ACC = 2.0 ** -15


def np8(t):
    return t.detach().cpu().numpy()


def gpu_bits(b):
    return W.bits_to_bf16(b).to(DEV)


def operand(rows, cols, seed, std=1.0):
    """A bf16 tensor quantised by the oracle: (codes, scales on the GPU, values in float64); above 4M
    values random codes and scales of a like size, which the oracle quantises too slowly."""
    if rows * cols > 1 << 22:
        r = np.random.default_rng(seed)
        c = r.integers(0, 256, (rows, cols // 2), dtype=np.uint8)
        s = r.integers(119, 126, (rows, cols // 32), dtype=np.uint8)
        return (torch.from_numpy(c).to(DEV), torch.from_numpy(R.store_scales(s)).to(DEV)), R.dequant(c, s)
    x = W.randn_bf16((rows, cols), seed, std).float()
    g = torch.Generator().manual_seed(seed + 1)
    x[:, torch.randperm(cols, generator=g)[: max(1, cols // 100)]] *= 20.0
    c, s = R.quant_bits(W.bf16_bits(x.to(torch.bfloat16)))
    return (torch.from_numpy(c).to(DEV), torch.from_numpy(R.store_scales(s)).to(DEV)), R.dequant(c, s)


@pytest.mark.parametrize("rows,cols", [(1, 128), (1, 4096), (3, 640), (17, 1920), (64, 14336), (1000, 384),
                                       (70000, 128)])
def test_quant_bit_exact(rows, cols):
    sp = need_sp()
    announce("quant_mxfp4", rows, cols)
    x = W.randn_bf16((rows, cols), rows + cols).float()
    x[0, ::7] *= 1000.0
    x[-1] = 0.0 if rows > 1 else x[-1]
    xb = x.to(torch.bfloat16)
    oc, os_ = R.quant_bits(W.bf16_bits(xb))
    c, s = sp.quant_mxfp4(xb.to(DEV))
    v = sp.dequant_mxfp4(c, s)
    torch.cuda.synchronize()
    assert np.array_equal(np8(s), R.store_scales(os_))
    assert np.array_equal(np8(c), oc)
    assert np.array_equal(bf16_to_f64(bits(v)), R.dequant(oc, os_))


def test_quant_every_bf16_pattern():
    """Every finite pattern as a block's maximum, beside values at and around every rounding boundary
    of its scale; then blocks with Inf and NaN."""
    sp = need_sp()
    announce("quant_mxfp4 every pattern")
    top = np.concatenate([np.arange(0, 0x7F80), np.arange(0x8000, 0xFF80)]).astype(np.uint16)
    v = bf16_to_f64(top)
    grid = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, 0.5, 1, 1.5, 2, 3, 4, 0.26, 0.24]) / 8
    near = W.bf16_bits(torch.from_numpy((np.abs(v)[:, None] * grid).astype(np.float32)).to(torch.bfloat16))
    b = np.zeros((len(top), 32), np.uint16)
    b[:, 0] = top
    b[:, 1:16] = near
    b[:, 16:31] = near | 0x8000
    odd = np.zeros((8, 32), np.uint16)
    for i, h in enumerate((0x7F80, 0xFF80, 0x7F81, 0xFFFF, 0x7FC0, 0x0000, 0x8000, 0x0001)):
        odd[i, 5 * i % 32] = h
        odd[i, 1] = 0x3F80 if i < 5 else odd[i, 1]
    b = np.concatenate([b, odd])
    b = np.concatenate([b, np.zeros((-len(b) % 4, 32), np.uint16)]).reshape(-1, 128)
    oc, os_ = R.quant_bits(b)
    c, s = sp.quant_mxfp4(gpu_bits(b))
    d = sp.dequant_mxfp4(c, s)
    torch.cuda.synchronize()
    assert np.array_equal(np8(s), R.store_scales(os_))
    assert np.array_equal(np8(c), oc)
    assert np.array_equal(bf16_to_f64(bits(d)), R.dequant(oc, os_), equal_nan=True)


# one token to many, around the kernels' tile edges; n and k odd multiples of their units
GEMM_SHAPES = [(1, 1, 128), (1, 14336, 4096), (1, 4096, 14336), (2, 16, 256), (3, 1000, 640), (5, 17, 1152),
               (15, 260, 512), (16, 4096, 4096), (17, 100, 896), (31, 333, 2048), (32, 512, 384), (33, 4096, 1408),
               (63, 257, 1024), (64, 4096, 14336), (65, 129, 768), (77, 4096, 14336), (100, 63, 16384),
               (128, 1024, 640), (129, 255, 384), (255, 6144, 512), (256, 4096, 4096), (257, 300, 1920),
               (333, 2000, 1024), (512, 512, 512), (1000, 1001, 640), (2049, 513, 384)]


@pytest.mark.parametrize("m,n,k", GEMM_SHAPES)
def test_gemm_against_oracle(m, n, k):
    sp = need_sp()
    announce("gemm_mxfp4", m, n, k)
    (xc, xs), x = operand(m, k, m + k)
    (wc, ws), w = operand(n, k, n + k + 7, 0.02)
    y = torch.full((m, n), float("nan"), dtype=torch.bfloat16, device=DEV)
    sp.gemm_mxfp4(xc, xs, wc, ws, out=y)
    torch.cuda.synchronize()
    ref, mag = R.gemm_ref(x, w)
    got = bf16_to_f64(bits(y))
    bad = ~(np.abs(got - ref) <= 2.0 ** -8 * np.abs(ref) + ACC * mag)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[0].tolist())
    y2 = sp.gemm_mxfp4(xc, xs, wc, ws)
    torch.cuda.synchronize()
    assert np.array_equal(bits(y), bits(y2))


# every configuration of the three kernels, at sizes around its tiles and with whole, half and
# few steps of K (the override picks it wherever it can run the call)
CONFIGS = ["stream,1", "stream,2", "stream,4", "stream,8"] + ["wave,%d" % i for i in range(6)] + \
    ["tiled,%d" % i for i in range(6)]


@pytest.mark.parametrize("config", CONFIGS)
def test_every_configuration(config, monkeypatch):
    sp = need_sp()
    monkeypatch.setenv("SP24_MX4", config)
    for m in ((1, 9, 16, 17, 33, 64) if config.startswith("stream") else (1, 31, 64, 65, 127, 129, 257)):
        for n, k in ((1, 128), (30, 640), (129, 1024), (256, 256), (260, 1408), (384, 2560)):
            announce(config, m, n, k)
            (xc, xs), x = operand(m, k, m + k)
            (wc, ws), w = operand(n, k, n + k + 7, 0.05)
            y = torch.full((m, n), float("nan"), dtype=torch.bfloat16, device=DEV)
            sp.gemm_mxfp4(xc, xs, wc, ws, out=y)
            torch.cuda.synchronize()
            ref, mag = R.gemm_ref(x, w)
            got = bf16_to_f64(bits(y))
            assert (np.abs(got - ref) <= 2.0 ** -8 * np.abs(ref) + ACC * mag).all(), (m, n, k)
            if n % 2:
                continue
            f = n // 2
            ref, err = R.gated_ref(x, w)
            err = ACC * err + 2.0 ** -16 * np.abs(ref)
            h = sp.gated_mxfp4(xc, xs, wc, ws)
            torch.cuda.synchronize()
            assert (np.abs(bf16_to_f64(bits(h)) - ref) <= 2.0 ** -8 * np.abs(ref) + err).all(), (m, n, k)
            if f % 128 == 0:
                c, s = sp.gated_mxfp4(xc, xs, wc, ws, quantise=True)
                torch.cuda.synchronize()
                check_mx4_output(c, s, ref, err, (m, n, k))


def test_gemm_extreme_scales_and_nan():
    """Scales from 2^-127 to 2^100 with products in range, and one row of X and one of W with a NaN block."""
    sp = need_sp()
    for m, n, k in ((3, 40, 640), (40, 70, 1024), (300, 300, 640)):
        announce("gemm_mxfp4 scales", m, n, k)
        r = np.random.default_rng(m)
        xc, wc = (r.integers(0, 256, (a, k // 2)).astype(np.uint8) for a in (m, n))
        xs = r.integers(0, 60, (m, k // 32)).astype(np.uint8)
        ws = r.integers(160, 228, (n, k // 32)).astype(np.uint8)
        xs[0, 0] = 0
        xs[m - 1, k // 64] = 255
        ws[n // 2, 1] = 255
        ref, mag = R.gemm_ref(R.dequant(xc, xs), R.dequant(wc, ws))
        y = sp.gemm_mxfp4(torch.from_numpy(xc).to(DEV), torch.from_numpy(R.store_scales(xs)).to(DEV),
                          torch.from_numpy(wc).to(DEV), torch.from_numpy(R.store_scales(ws)).to(DEV))
        torch.cuda.synchronize()
        got = bf16_to_f64(bits(y))
        assert np.array_equal(np.isnan(got), np.isnan(ref))
        ok = np.isnan(ref) | (np.abs(got - ref) <= 2.0 ** -8 * np.abs(ref) + ACC * mag + 2.0 ** -120)
        assert ok.all(), int((~ok).sum())


GATED_SHAPES = [(1, 128, 128), (1, 14336, 4096), (2, 384, 640), (7, 1000, 384), (16, 640, 1024), (17, 33, 512),
                (33, 256, 1152), (64, 4096, 640), (65, 1, 256), (100, 384, 1920), (128, 2048, 512), (200, 513, 384),
                (300, 1280, 896), (1025, 640, 640)]


def check_mx4_output(codes, stored, h, err, what):
    """codes/scales on the GPU hold h (float64) as the quantiser rounds it, where h may be off by err:
    each block's scale is that of a maximum within err, each value within half a step (and err)."""
    rows, cols = h.shape
    s = R.load_scales(np8(stored), rows, cols)
    b, d = np.abs(h.reshape(rows, -1, 32)), err.reshape(rows, -1, 32)
    lo = R.block_scale_bytes(np.maximum(b - d, 0).reshape(rows, cols)).astype(int)
    hi = R.block_scale_bytes((b + d).reshape(rows, cols)).astype(int)
    zero = ((b - d).max(-1) <= 0)  # a maximum that may be 0: scale 1 as well
    assert (((lo <= s) & (s <= hi)) | (zero & ((s == 127) | (s <= hi)))).all(), what
    scale = R.scale_values(s)[..., None]
    got = R.dequant(np8(codes), s).reshape(rows, -1, 32)
    want = np.clip(h.reshape(rows, -1, 32), -6 * scale, 6 * scale)
    a = np.abs(want) / scale
    step = np.where(a < 2, 0.5, np.where(a < 4, 1.0, 2.0)) * scale
    # at a binade's lower edge the step below is half: the larger of the two bounds both sides
    assert (np.abs(got - want) <= 0.5 * step * (1 + 1e-12) + d).all(), what


@pytest.mark.parametrize("m,f,k", GATED_SHAPES)
def test_gated_against_oracle(m, f, k):
    sp = need_sp()
    announce("gated_mxfp4", m, f, k)
    (xc, xs), x = operand(m, k, m + k + 1)
    (wc, ws), w = operand(2 * f, k, f + k + 9, 0.05)
    h = sp.gated_mxfp4(xc, xs, wc, ws)
    torch.cuda.synchronize()
    ref, err = R.gated_ref(x, w)
    err = ACC * err + 2.0 ** -16 * np.abs(ref)
    got = bf16_to_f64(bits(h))
    bad = ~(np.abs(got - ref) <= 2.0 ** -8 * np.abs(ref) + err)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[0].tolist())
    if f % 128 == 0:
        c, s = sp.gated_mxfp4(xc, xs, wc, ws, quantise=True)
        torch.cuda.synchronize()
        check_mx4_output(c, s, ref, err, (m, f, k))


def test_gated_nan_rows():
    """A NaN block of one token makes that token's h NaN (scale byte 255 in the MXFP4 form), no other's."""
    sp = need_sp()
    for m in (3, 70, 300):
        announce("gated_mxfp4 nan", m)
        (xc, xs), x = operand(m, 256, 5)
        s = R.load_scales(np8(xs), m, 256)
        s[1, 2] = 255
        xs = torch.from_numpy(R.store_scales(s)).to(DEV)
        (wc, ws), w = operand(256, 256, 6, 0.05)
        h = sp.gated_mxfp4(xc, xs, wc, ws)
        c, hs = sp.gated_mxfp4(xc, xs, wc, ws, quantise=True)
        torch.cuda.synchronize()
        nan = np.isnan(bf16_to_f64(bits(h)))
        assert nan[1].all() and not np.delete(nan, 1, 0).any()
        b = R.load_scales(np8(hs), m, 128)
        assert (b[1] == 255).all() and (np.delete(b, 1, 0) != 255).all() and not np8(c)[1].any()


@pytest.mark.parametrize("m,d,f", [(1, 256, 384), (16, 640, 512), (50, 128, 1024), (300, 512, 640)])
def test_ffn_is_its_three_calls(m, d, f):
    sp = need_sp()
    announce("ffn_mxfp4", m, d, f)
    x, r = (W.randn_bf16((m, d), seed).to(DEV) for seed in (m, d))
    w = W.randn_bf16((d,), f).to(DEV)
    gu = sp.quant_mxfp4(W.randn_bf16((2 * f, d), 3, 0.05).to(DEV))
    dn = sp.quant_mxfp4(W.randn_bf16((d, f), 4, 0.05).to(DEV))
    for res in (r, None):
        y, ro = sp.ffn_mxfp4(x, w, *gu, *dn, residual=res, eps=1e-5)
        q, s, ro2 = sp.rmsnorm(x, w, sp.NORM_MXFP4, residual=res, eps=1e-5)
        y2 = sp.gemm_mxfp4(*sp.gated_mxfp4(q, s, *gu, quantise=True), *dn)
        torch.cuda.synchronize()
        assert np.array_equal(bits(y), bits(y2))
        assert (ro is None and ro2 is None) if res is None else np.array_equal(bits(ro), bits(ro2))


def test_calls_on_another_stream_and_in_a_graph():
    """The block on a side stream, then captured and replayed with new inputs between eager calls."""
    sp = need_sp()
    m, d, f = 5, 512, 640
    announce("ffn_mxfp4 stream and graph")
    gu = sp.quant_mxfp4(W.randn_bf16((2 * f, d), 3, 0.05).to(DEV))
    dn = sp.quant_mxfp4(W.randn_bf16((d, f), 4, 0.05).to(DEV))
    w = W.randn_bf16((d,), 9).to(DEV)
    xs = [W.randn_bf16((m, d), 20 + i).to(DEV) for i in range(5)]
    ws = torch.empty(sp.ffn_mxfp4_workspace_size(m, d, f), dtype=torch.uint8, device=DEV)
    want = [sp.ffn_mxfp4(x, w, *gu, *dn)[0].clone() for x in xs]
    x, y = xs[0].clone(), torch.empty(m, d, dtype=torch.bfloat16, device=DEV)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        sp.ffn_mxfp4(x, w, *gu, *dn, out=y, ws=ws)
    st.synchronize()
    assert torch.equal(y.view(torch.int16), want[0].view(torch.int16))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sp.ffn_mxfp4(x, w, *gu, *dn, out=y, ws=ws)
    for i in range(5):
        x.copy_(xs[i])
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y.view(torch.int16), want[i].view(torch.int16)), i
        sp.ffn_mxfp4(xs[(i + 1) % 5], w, *gu, *dn)


def test_scales_past_4gib():
    """A weight whose codes pass 2^32 bytes: rows at both ends against the oracle."""
    sp = need_sp()
    rows, cols = 70000, 131072
    announce("gemm_mxfp4 long weight", rows, cols)
    codes = torch.randint(0, 256, (rows, cols // 2), dtype=torch.uint8, device=DEV,
                          generator=torch.Generator(device=DEV).manual_seed(1))
    scales = torch.randint(118, 128, (rows * cols // 32,), dtype=torch.uint8, device=DEV,
                           generator=torch.Generator(device=DEV).manual_seed(2))
    (xc, xs), x = operand(2, cols, 3)
    y = sp.gemm_mxfp4(xc, xs, codes, scales)
    pick = [0, 1, 33333, rows - 2, rows - 1]
    idx = sp.mxfp4_scale_index(1, cols)[0]
    b, width = (idx // 4) // 4, 4
    at = 4 * (4 * rows * b[None] + torch.tensor(pick)[:, None] * width + (idx // 4) % 4) + idx % 4
    s = np8(scales[at.to(DEV)])
    w = R.dequant(np8(codes[pick]), s)
    got = bf16_to_f64(bits(y))[:, pick]
    ref, mag = R.gemm_ref(x, w)
    # k = 131072: 2048 accumulations of an instruction, 8 times those ACC was derived for
    assert (np.abs(got - ref) <= 2.0 ** -8 * np.abs(ref) + 8 * ACC * mag).all()


def test_binding_refusals():
    """What the binding refuses on GPU tensors: types, shapes, strides, devices, outputs, sizes."""
    sp = need_sp()
    announce("mxfp4 binding refusals")
    x = torch.zeros(4, 256, dtype=torch.bfloat16, device=DEV)
    w = torch.zeros(256, dtype=torch.bfloat16, device=DEV)
    c, s = sp.quant_mxfp4(x)
    wide = torch.zeros(4, 512, dtype=torch.bfloat16, device=DEV)[:, :256]
    for bad, err in ((x.float(), TypeError), (x.cpu(), ValueError), (x[0], ValueError), (wide, ValueError),
                     (x[:, :200].contiguous(), ValueError), (x[:0], sp.Sp24Error), (None, TypeError)):
        with pytest.raises(err):
            sp.quant_mxfp4(bad)
    for kw in (dict(out=c.view(8, 64)), dict(out=c.int()), dict(scales=s[:-1]), dict(out=c.cpu())):
        with pytest.raises((ValueError, TypeError)):
            sp.quant_mxfp4(x, **kw)
    c2, s2 = sp.quant_mxfp4(torch.zeros(6, 384, dtype=torch.bfloat16, device=DEV))
    for args in ((c, s, c2, s2), (c, s[:-1], c, s), (c[:, :60].contiguous(), s, c, s), (c.cpu(), s, c, s)):
        with pytest.raises(ValueError):
            sp.gemm_mxfp4(*args)
    for args, kw in (((c, s, c[:3].contiguous(), s[:24].contiguous()), {}), ((c, s, c, s), dict(quantise=True)),
                     ((c, s, c, s), dict(out_scales=s)), ((c, s, c, s), dict(out=x))):
        with pytest.raises(ValueError):
            sp.gated_mxfp4(*args, **kw)
    for kw in (dict(kind=9), dict(residual=x[:2]), dict(residual_out=x), dict(kind=sp.NORM_FP8_GROUPS, group=100),
               dict(scales=torch.zeros(4, device=DEV)), dict(kind=sp.NORM_MXFP4, out=x),
               dict(kind=sp.NORM_FP8_ROWS, scales=torch.zeros(3, device=DEV))):
        with pytest.raises((ValueError, TypeError)):
            sp.rmsnorm(x, w, **kw)
    with pytest.raises(ValueError):
        sp.rmsnorm(x, w[:128])
    for eps in (0.0, float("nan")):
        with pytest.raises(sp.Sp24Error) as e:
            sp.rmsnorm(x, w, eps=eps)
        assert e.value.status == -7
    with pytest.raises(sp.Sp24Error) as e:
        sp.rmsnorm(x, w, residual=wide.contiguous(), residual_out=x)   # an output over an input
    assert e.value.status == -8
    with pytest.raises(ValueError):
        sp.ffn_mxfp4(x, w, c, s, c, s)
