"""The example's stack against float64: what its blocks add to the tokens, not the stream, most of which
is the tokens themselves."""
import numpy as np
import pytest
import torch

import workloads as W
from gpu_helpers import DEV, announce, bits, need_sp
from mxfp4_stack import FAR, SIZES, contribution, distance, weights
from oracle.sp24_ref import bf16_to_f64

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("layers,d,f,m", SIZES)
def test_contribution(layers, d, f, m):
    sp = need_sp()
    from bf16_gemm_linear_amd import mxfp4_ffn
    announce("mxfp4 stack", layers, d, f, m)
    x = W.randn_bf16((m, d), 1)
    blocks, gen = [], torch.Generator(DEV).manual_seed(1)
    for gu, dn in weights(layers, d, f):
        b = mxfp4_ffn.Block(d, f, gen, torch.device(DEV))
        b.gate_up, b.down = W.bits_to_bf16(gu).to(DEV), W.bits_to_bf16(dn).to(DEV)
        b.gu, b.dn = sp.quant_mxfp4(b.gate_up), sp.quant_mxfp4(b.down)
        blocks.append(b)
    s = mxfp4_ffn.Stack(blocks, m, d, f, torch.device(DEV))
    s.x.copy_(x)
    s.mxfp4()
    graph = mxfp4_ffn.captured(s.mxfp4)
    torch.cuda.synchronize()
    start = bf16_to_f64(W.bf16_bits(x))
    want = contribution(start, weights(layers, d, f))
    assert distance(bf16_to_f64(bits(s.r)) - start, want) < FAR
    for i in range(3):  # a replay computes it anew, whatever its buffers hold
        s.r.fill_(float(i))
        for y in s.y:
            y.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert distance(bf16_to_f64(bits(s.r)) - start, want) < FAR
