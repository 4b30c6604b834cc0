"""The MXFP4 quantiser past the units that its largest grid takes in one go (131072 of 128 values), and
the way back: bit for bit, with a remainder, and rows whose last block of scales is narrower."""
import numpy as np
import pytest
import torch

import workloads as W
from gpu_helpers import DEV, announce, bits, need_sp
from oracle import mxfp4_ref as R
from oracle.sp24_ref import bf16_to_f64
from test_gpu_mxfp4 import np8

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,cols", [(140001, 128), (9001, 2176), (37003, 1152)])
def test_quant_beyond_one_grid(rows, cols):
    sp = need_sp()
    announce("quant_mxfp4", rows, cols)
    assert rows * cols // 128 > 8192 * 16
    x = W.randn_bf16((rows, cols), rows).float()
    x *= torch.exp2(torch.arange(rows) % 61 - 30.0)[:, None]  # a row's scales are its own
    xb = x.to(torch.bfloat16)
    c, s = sp.quant_mxfp4(xb.to(DEV))
    v = sp.dequant_mxfp4(c, s)
    torch.cuda.synchronize()
    c, s, v = np8(c), R.load_scales(np8(s), rows, cols), bits(v)
    edge = 8192 * 16 * 128 // cols  # the row that the second go begins in
    for a, b in ((0, 2000), (edge - 1000, edge + 1000), (rows - 2000, rows)):
        oc, os_ = R.quant_bits(W.bf16_bits(xb[a:b]))
        assert np.array_equal(s[a:b], os_)
        assert np.array_equal(c[a:b], oc)
        assert np.array_equal(bf16_to_f64(v[a:b]), R.dequant(oc, os_))
    # every other row: its values within half a step of its own scale
    f, amax = xb.float().numpy(), xb.float().abs().view(rows, -1, 32).amax(-1).numpy()
    assert np.array_equal(s.astype(np.int32) - 127, np.frexp(np.where(amax > 0, amax, 4.0))[1] - 3)
    step = np.ldexp(np.float32(1), s.astype(np.int32) - 127).repeat(32, axis=1)
    assert (np.abs(W.bits_to_bf16(v).float().numpy() - f) <= 2 * step).all()
