"""Every configuration of the MXFP4 products, by name and with no other in its place, in every output
that it has, and the ones that the feed-forward block takes at its own sizes.

Sizes: several tile columns, several steps of K for every wave that shares it (k = 2560 and 4096 in
whole blocks of scales, 1408 and 2176 with a half last step), token tiles whole and not.  Tolerances
are test_gpu_mxfp4's: k <= 4096 is at most 64 + 64 roundings, 2^-16 of the sum of magnitudes, under its
2^-15."""
import numpy as np
import pytest
import torch

from gpu_helpers import announce, bits, need_sp
from oracle import mxfp4_ref as R
from oracle.sp24_ref import bf16_to_f64
from test_gpu_mxfp4 import ACC, check_mx4_output, np8, operand

pytestmark = pytest.mark.gpu

STREAM = {1: (False, False), 2: (True, False), 4: (True, True), 8: (True, True)}  # gated in bf16, in MXFP4
CONFIGS = [("stream,%d" % i, *o) for i, o in STREAM.items()] + [("wave,%d" % i, i < 5, i < 5) for i in range(6)] + \
    [("tiled,%d" % i, i < 4, i < 4) for i in range(6)]


def tokens(config):
    if config == "stream,8":
        return (1, 8, 9, 16)
    return (3, 8, 12, 16, 29, 50, 64) if config.startswith("stream") else (16, 100, 260)


@pytest.mark.parametrize("config,bf16,mx", CONFIGS)
def test_named_configuration(config, bf16, mx, monkeypatch):
    sp = need_sp()
    monkeypatch.setenv("SP24_MX4", config + "!")
    for f, k in ((384, 2560), (640, 1408), (256, 4096), (130, 2176)):
        (wc, ws), w = operand(2 * f, k, f + k + 9, 0.05)
        for m in tokens(config):
            announce(config, m, f, k)
            (xc, xs), x = operand(m, k, m + k + 1)
            y = sp.gemm_mxfp4(xc, xs, wc, ws)
            torch.cuda.synchronize()
            ref, mag = R.gemm_ref(x, w)
            assert (np.abs(bf16_to_f64(bits(y)) - ref) <= 2.0 ** -8 * np.abs(ref) + ACC * mag).all(), (m, f, k)
            ref, err = R.gated_ref(x, w)
            err = ACC * err + 2.0 ** -16 * np.abs(ref)
            if bf16:
                h = sp.gated_mxfp4(xc, xs, wc, ws)
                torch.cuda.synchronize()
                assert (np.abs(bf16_to_f64(bits(h)) - ref) <= 2.0 ** -8 * np.abs(ref) + err).all(), (m, f, k)
            if mx and f % 128 == 0:
                c, s = sp.gated_mxfp4(xc, xs, wc, ws, quantise=True)
                torch.cuda.synchronize()
                check_mx4_output(c, s, ref, err, (m, f, k))


def test_an_output_that_a_configuration_lacks(monkeypatch):
    sp = need_sp()
    (wc, ws), _ = operand(512, 256, 1)
    (xc, xs), _ = operand(20, 256, 2)
    for config, call in (("wave,5!", lambda: sp.gated_mxfp4(xc, xs, wc, ws)),
                         ("stream,2!", lambda: sp.gated_mxfp4(xc, xs, wc, ws, quantise=True)),
                         ("stream,8!", lambda: sp.gemm_mxfp4(xc, xs, wc, ws))):
        monkeypatch.setenv("SP24_MX4", config)
        with pytest.raises(sp.Sp24Error):
            call()


@pytest.mark.parametrize("m", [9, 16, 77, 1000, 2047])
def test_gated_to_mxfp4_at_the_blocks_sizes(m):
    """4096 x 14336, the kernel that the planner takes; some tokens of each tile are compared."""
    sp = need_sp()
    f, k = 14336, 4096
    announce("gated_mxfp4 quantise", m, f, k)
    (xc, xs), x = operand(m, k, m)
    (wc, ws), w = operand(2 * f, k, 5)
    c, s = sp.gated_mxfp4(xc, xs, wc, ws, quantise=True)
    h = sp.gated_mxfp4(xc, xs, wc, ws)
    torch.cuda.synchronize()
    pick = np.unique(np.r_[0:min(m, 9), np.arange(31, m, 97), max(0, m - 3):m])
    ref, err = R.gated_ref(x[pick], w)
    err = ACC * err + 2.0 ** -16 * np.abs(ref)
    part = torch.from_numpy(R.store_scales(R.load_scales(np8(s), m, f)[pick]))
    at = torch.from_numpy(pick).to(c.device)
    check_mx4_output(c[at], part, ref, err, (m, f, k))
    assert (np.abs(bf16_to_f64(bits(h[at])) - ref) <= 2.0 ** -8 * np.abs(ref) + err).all()
