"""What the stack's measure tells apart, on the CPU: a block that adds nothing, one of the wrong sign,
one whose norm or scales are off, in any layer, are all further than the kernels may be."""
import numpy as np
import pytest

import workloads as W
from mxfp4_stack import FAR, SIZES, contribution, distance, weights
from oracle.sp24_ref import bf16_to_f64


@pytest.mark.parametrize("layers,d,f,m", SIZES)
def test_planted_mistakes_are_far(layers, d, f, m):
    x = bf16_to_f64(W.bf16_bits(W.randn_bf16((m, d), 1)))
    blocks = weights(layers, d, f)
    want = contribution(x, blocks)
    assert 0.3 < np.linalg.norm(want) / np.linalg.norm(x) < 5 * layers  # the blocks count beside the tokens
    for layer in range(layers):
        for name, wrong in (("nothing", lambda y: 0 * y), ("sign", lambda y: -y), ("half", lambda y: y / 2),
                            ("double", lambda y: 2 * y), ("another token's", lambda y: np.roll(y, 1, 0) if m > 1 else -y),
                            ("another column's", lambda y: np.roll(y, 32, 1))):
            got = contribution(x, blocks, plant=lambda i, y: wrong(y) if i == layer else y)
            assert distance(got, want) > 2 * FAR, (layer, name)


@pytest.mark.parametrize("layers,d,f,m", SIZES)
def test_quantisation_costs_what_its_steps_say(layers, d, f, m):
    """Against the same blocks unquantised: more than the kernels may differ by, and for one layer at most
    0.36: an operand is off by 1/8 of itself rms at most, h by the gate's error times g silu'(g) / silu(g)
    (mean square below 1.5 over unit gates, weighted by h^2) and by the up value's: sqrt((2 1.5 + 2 + 2) / 64)
    = 0.33, a tenth more for few tokens."""
    x = bf16_to_f64(W.bf16_bits(W.randn_bf16((m, d), 1)))
    blocks = weights(layers, d, f)
    far = distance(contribution(x, blocks), contribution(x, blocks, quantised=False))
    assert FAR < far < (0.36 if layers == 1 else 1.0), far
