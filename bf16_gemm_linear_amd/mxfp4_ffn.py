"""Example: a stack of pre-norm feed-forward blocks with MXFP4 weights, as a server runs it.

    python -m bf16_gemm_linear_amd.mxfp4_ffn [--layers 4] [--d 4096] [--f 14336] [--prefill 1024] [--batch 16]

Quantises synthetic bf16 weights once (`quant_mxfp4`), sends a prompt of `--prefill` tokens through
the stack, then decodes `--batch` tokens a step from one captured HIP graph whose every launch is
this library's: per layer one `ffn_mxfp4` (RMS norm with residual addition and MXFP4 output, gated
product with MXFP4 output, down product), the residual carried in place, and at the end `rmsnorm`
in bf16.  The same stack in bf16 with PyTorch's own operators runs beside it.  Prints one JSON
object: milliseconds of each, weight bytes, and the relative error of MXFP4 against bf16 (what 4-bit
weights and activations cost on random data, layer after layer, not an error of the kernels: those
agree with the same blocks in float64 on the same 4-bit values).
"""
from __future__ import annotations

import argparse
import json
import time

import torch
import torch.nn.functional as F

import bf16_gemm_linear_amd as sp


class Block:
    """One layer: the norm's weight and the gate-over-up and down weights in both forms."""

    def __init__(self, d, f, gen, device):
        def weight(n, k):
            return torch.empty(n, k, dtype=torch.bfloat16, device=device).normal_(0, 0.02, generator=gen)

        self.norm = torch.ones(d, dtype=torch.bfloat16, device=device)
        self.gate_up, self.down = weight(2 * f, d), weight(d, f)
        self.gu, self.dn = sp.quant_mxfp4(self.gate_up), sp.quant_mxfp4(self.down)


class Stack:
    """`h` is a layer's output, `r` the residual it has not been added to yet."""

    def __init__(self, blocks, m, d, f, device):
        self.blocks = blocks
        self.x = torch.empty(m, d, dtype=torch.bfloat16, device=device)  # the caller's tokens
        self.r = torch.empty_like(self.x)
        self.y = [torch.empty_like(self.x), torch.empty_like(self.x)]  # a block's output is not its input
        self.out = torch.empty_like(self.x)
        self.final = torch.ones(d, dtype=torch.bfloat16, device=device)
        self.ws = torch.empty(sp.ffn_mxfp4_workspace_size(m, d, f), dtype=torch.uint8, device=device)

    def mxfp4(self):
        self.r.zero_()
        h = self.x
        for i, b in enumerate(self.blocks):
            h, _ = sp.ffn_mxfp4(h, b.norm, *b.gu, *b.dn, residual=self.r, out=self.y[i % 2], residual_out=self.r,
                                ws=self.ws)
        sp.rmsnorm(h, self.final, residual=self.r, out=self.out, residual_out=self.r)
        return self.out

    def bf16(self):
        r = self.x
        d = r.shape[1]
        for b in self.blocks:
            v = F.rms_norm(r, (d,), b.norm, 1e-6)
            gate, up = F.linear(v, b.gate_up).chunk(2, dim=1)
            r = r + F.linear(F.silu(gate) * up, b.down)
        return F.rms_norm(r, (d,), self.final, 1e-6)


def milliseconds(call, reps=20):
    call()
    torch.cuda.synchronize()
    t = time.perf_counter()
    for _ in range(reps):
        call()
    torch.cuda.synchronize()
    return (time.perf_counter() - t) / reps * 1e3


def captured(call):
    """The call as a HIP graph."""
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):  # a first run outside the capture: allocations, code objects
        call()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    return graph


def main(argv=None):
    p = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    p.add_argument("--layers", type=int, default=4)
    p.add_argument("--d", type=int, default=4096)
    p.add_argument("--f", type=int, default=14336)
    p.add_argument("--prefill", type=int, default=1024)
    p.add_argument("--batch", type=int, default=16)
    a = p.parse_args(argv)
    device = torch.device("cuda")
    gen = torch.Generator(device).manual_seed(7)
    blocks = [Block(a.d, a.f, gen, device) for _ in range(a.layers)]
    got = {"layers": a.layers, "d": a.d, "f": a.f,
           "weight_bytes_bf16": sum(2 * (b.gate_up.numel() + b.down.numel()) for b in blocks),
           "weight_bytes_mxfp4": sum(t.numel() for b in blocks for t in (*b.gu, *b.dn))}
    for name, m in (("prefill", a.prefill), ("decode", a.batch)):
        s = Stack(blocks, m, a.d, a.f, device)
        s.x.normal_(generator=gen)
        want = s.bf16().float()
        y = s.mxfp4().float()
        got[name] = {"tokens": m, "mxfp4_ms": milliseconds(s.mxfp4), "bf16_ms": milliseconds(s.bf16),
                     "relative_error": float((y - want).norm() / want.norm())}
        if name == "decode":
            graph = captured(s.mxfp4)
            for _ in range(3):  # new tokens into the same buffers, one replay a step
                s.x.normal_(generator=gen)
                graph.replay()
                replayed = s.out.clone()
                assert torch.equal(replayed, s.mxfp4()), "the graph's output differs from the calls'"
            got[name]["mxfp4_graph_ms"] = milliseconds(graph.replay)
    print(json.dumps(got))
    return got


if __name__ == "__main__":
    main()
