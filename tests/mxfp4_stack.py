"""The example's stack of MXFP4 feed-forward blocks in float64 (quantised by the oracle), and how far a
stack's contribution, the residual less the tokens it began with, is from another's."""
import numpy as np

import workloads as W
from oracle import mxfp4_ref as R
from oracle.sp24_ref import bf16_to_f64

# layers, d, f, tokens
SIZES = [(1, 512, 1280, 130), (1, 512, 1280, 5), (1, 128, 128, 1), (3, 1024, 640, 33), (3, 1024, 640, 64)]
# Relative error of a contribution that the kernels may have.  They and this module round the same
# numbers, which differ by the kernels' fp32: where one lies so near a code's boundary its code is the
# next one, a step of at most 1/2 of the value, 1/3 rms over where boundaries lie.  With boundaries
# a quarter of a value apart and an error of up to 2^-12 in h (2^-15 of the sum of magnitudes, some
# eight times |h|), 2^-9 of the codes: sqrt(2^-9) / 3 = 0.015.  From the second layer the bf16
# residual, whose roundings follow y's, moves v by up to 2^-9, 2^-6 of the codes, 0.042 for each of
# the two layers that it feeds: 0.06 together.
FAR = 0.08


def weights(layers, d, f):
    """bf16 gate-over-up and down weights by which a block adds about as much as it is given (unit
    gate and up values, h of about 0.6, unit outputs), as bit patterns."""
    return [(W.bf16_bits(W.randn_bf16((2 * f, d), 10 + i, d ** -0.5)), W.bf16_bits(W.randn_bf16((d, f), 20 + i, 1.7 * f ** -0.5)))
            for i in range(layers)]


def rounded(v):
    """float64 -> the values of bf16, nearest even."""
    import torch
    return bf16_to_f64(W.bf16_bits(torch.from_numpy(v).to(torch.float32).to(torch.bfloat16)))


def normed(t):
    return t / np.sqrt((t * t).mean(-1, keepdims=True) + 1e-6)


def stored(v):
    """What the MXFP4 form of v stands for."""
    return R.dequant(*R.quant(v))


def contribution(x, blocks, quantised=True, plant=lambda i, y: y):
    """Residual after the stack less x (float64); `plant` alters layer i's output."""
    q = stored if quantised else (lambda v: v)
    r, h = np.zeros_like(x), x
    for i, (gu, dn) in enumerate(blocks):
        gu, dn = q(bf16_to_f64(gu)), q(bf16_to_f64(dn))
        t = h + r
        r, f = rounded(t), gu.shape[0] // 2
        gate_up = q(normed(t)) @ gu.T
        h = rounded(plant(i, q(R.silu(gate_up[:, :f]) * gate_up[:, f:]) @ dn.T))
    return rounded(h + r) - x


def distance(a, b):
    return np.linalg.norm(a - b) / np.linalg.norm(b)
