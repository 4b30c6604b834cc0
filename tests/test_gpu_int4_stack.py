"""The operators in a row, as a server of experts runs them: per layer the RMS norm with residual addition,
the router's product in bf16, the routing, the experts' block over integer 4-bit weights; at the end a
4-bit output projection.  Each step is held to 64 bits on the tensors that the step before it gave, and a
captured graph of the whole, replayed on new tokens, to the eager calls bit for bit."""
import numpy as np
import pytest
import torch

import workloads as W
from gpu_helpers import DEV, announce, need_sp
from oracle import int4_ref as R
from test_gpu_experts import experts, reference
from test_gpu_int4 import f64, product, tolerance, weight

pytestmark = pytest.mark.gpu
D, F, E, TOP, LAYERS, VOCAB = 256, 192, 16, 4, 2, 1000


class Model:
    def __init__(self, group, zeros):
        self.layers = [experts(E, D, F, group, zeros, 40 + i) for i in range(LAYERS)]
        self.router = [W.randn_bf16((E, D), 70 + i, 0.1).to(DEV) for i in range(LAYERS)]
        self.bias = [0.05 * torch.randn(E, generator=torch.Generator().manual_seed(i)).to(DEV) for i in range(LAYERS)]
        self.norm = torch.ones(D, dtype=torch.bfloat16, device=DEV)
        self.head = weight(VOCAB, D, group, zeros, 90)

    def run(self, sp, x, keep):
        """`keep` gets every step's tensors."""
        r, h = torch.zeros_like(x), x
        for (args, _, _), w, b in zip(self.layers, self.router, self.bias):
            v, _, r = sp.rmsnorm(h, self.norm, sp.NORM_BF16, residual=r)
            l = sp.dense_gemm(v, w)
            ids, wt = sp.route(l, TOP, kind=sp.ROUTE_SIGMOID, bias=b, groups=4, top_groups=2, group_best=2, factor=2.0)
            h = sp.experts_int4(v, ids, wt, *args[:4], gu_zeros=args[4], down_zeros=args[5])
            keep.append((v, l, ids, wt, h))
        v, _, _ = sp.rmsnorm(h, self.norm, sp.NORM_BF16, residual=r)
        y = sp.gemm_int4(v, *self.head[0])
        keep.append((v, y))
        return y


@pytest.mark.parametrize("tokens", [1, 3, 24, 180, 700])
@pytest.mark.parametrize("group,zeros", [(64, True), (32, False)])
def test_stack(tokens, group, zeros):
    sp = need_sp()
    announce("int4 stack", tokens, group, zeros)
    m = Model(group, zeros)
    x = W.randn_bf16((tokens, D), tokens).to(DEV)
    keep = []
    m.run(sp, x, keep)
    torch.cuda.synchronize()
    for (_, gu, dn), b, (v, l, ids, wt, h) in zip(m.layers, m.bias, keep):
        want, ww = R.route(l.double().cpu().numpy(), TOP, sigmoid=True, bias=b.double().cpu().numpy(), groups=4,
                           top_groups=2, group_best=2, factor=2.0)
        assert np.array_equal(ids.cpu().numpy(), want)
        assert (np.abs(f64(wt) - ww) <= 2.0 ** -20 * ww).all()
        ref, tol = reference(f64(v), ids.cpu().numpy(), f64(wt), gu, dn, F)
        assert (np.abs(f64(h) - ref) <= tol).all()
    v, y = keep[-1]
    _, w, q, s, z = m.head
    ref = product(f64(v), w)
    assert (np.abs(f64(y) - ref) <= tolerance(f64(v), w, q, s, z, ref)).all()


@pytest.mark.parametrize("tokens", [1, 24, 400])
def test_stack_from_a_graph(tokens):
    sp = need_sp()
    announce("int4 stack graph", tokens)
    m = Model(64, True)
    x = torch.zeros(tokens, D, dtype=torch.bfloat16, device=DEV)
    m.run(sp, x, [])
    torch.cuda.synchronize()
    graph, kept = torch.cuda.CUDAGraph(), []
    with torch.cuda.graph(graph):
        y = m.run(sp, x, kept)
    for seed in range(3):
        x.copy_(W.randn_bf16((tokens, D), 5 + seed))
        graph.replay()
        torch.cuda.synchronize()
        got, eager = y.clone(), []
        assert torch.equal(got, m.run(sp, x, eager))
        assert all(torch.equal(a, b) for g, e in zip(kept, eager) for a, b in zip(g, e))
