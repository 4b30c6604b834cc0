"""The integer 4-bit oracle pinned to values worked out by hand, and to its own definition."""
import numpy as np
import pytest
import torch

import workloads as W
from oracle import int4_ref as R
from oracle.sp24_ref import bf16_to_f32


def bits(values):
    return W.bf16_bits(torch.tensor(values, dtype=torch.float64).to(torch.bfloat16))


def test_word_order():
    word = np.array([[1, 2, 3, 4, 5, 6, 7, 8]], np.uint8)
    # nibbles from the lowest: values 0 2 4 6 1 3 5 7
    assert R.pack(word).tolist() == [[0x31, 0x75, 0x42, 0x86]]
    q = np.random.default_rng(0).integers(0, 16, (3, 4, 96), dtype=np.uint8)
    assert np.array_equal(R.unpack(R.pack(q)), q)


def test_bf16_round_against_torch():
    r = np.random.default_rng(1)
    v = np.concatenate((r.standard_normal(5000) * np.exp2(r.integers(-40, 40, 5000)), [0.0, 1e-40, -3e-39, 2.0 ** -134]))
    f = v.astype(np.float32)
    assert np.array_equal(R.bf16_round(f.astype(np.float64)),
                          torch.from_numpy(f).to(torch.bfloat16).double().numpy())


def test_symmetric_by_hand():
    w = np.zeros((1, 32))
    w[0, :6] = [7.0, -7.0, 0.5, 1.5, -2.5, 3.49]
    q, s, z = R.quant(bits(w), 32, False)
    assert s.tolist() == [[1.0]] and z is None
    assert q[0, :6].tolist() == [15, 1, 8, 10, 6, 11]  # ties to even: 0.5 -> 0, 1.5 -> 2, -2.5 -> -2


def test_zero_points_by_hand():
    w = np.zeros((2, 32))
    w[0, :4] = [-5.0, 10.0, 0.0, 2.4]
    w[1] = 3.0  # all positive: the range reaches down to 0
    q, s, z = R.quant(bits(w), 32, True)
    assert s[:, 0].tolist() == [1.0, 0.2001953125] and z[:, 0].tolist() == [5, 0]
    assert q[0, :4].tolist() == [0, 15, 5, 7] and q[1].tolist() == [15] * 32


@pytest.mark.parametrize("zeros", [False, True])
def test_zero_and_nonfinite_groups(zeros):
    w = np.zeros((1, 96))
    w[0, 40], w[0, 70] = np.inf, np.nan
    q, s, z = R.quant(bits(w), 32, zeros)
    assert s[0, 0] == 1.0 and np.isnan(s[0, 1:]).all()
    assert (q[0, 32:] == 8).all() and (R.dequant(q, s, z)[0, :32] == 0).all()


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_error_is_half_a_step(group, zeros):
    b = W.bf16_bits(W.randn_bf16((16, 256), 3, 0.02))
    q, s, z = R.quant(b, group, zeros)
    d = np.abs(R.dequant(q, s, z) - bf16_to_f32(b))
    # s is rounded by 2^-9 of it, so the ends of the range lie up to 15 2^-8 steps outside
    assert (d <= np.repeat(s, group, 1) * (0.5 + 15 * 2.0 ** -8)).all()


def test_route_by_hand():
    l = [[1.0, 3.0, 3.0, 2.0]]
    ids, w = R.route(l, 3)
    assert ids.tolist() == [[1, 2, 3]]
    assert np.allclose(w, np.array([1, 1, np.exp(-1)]) / (2 + np.exp(-1)))
    ids, w = R.route(l, 2, renormalise=False, factor=2.0)
    assert np.allclose(w, 2 * np.exp(3) / (np.exp(1) + 2 * np.exp(3) + np.exp(2)))
    ids, _ = R.route(l, 2, sigmoid=True, bias=[1.0, 0.0, 0.0, 0.0])
    assert ids.tolist() == [[0, 1]]
    # groups {0, 1}, {2, 3}: best one 3 and 3 (the first wins), best two scores: the second
    assert R.route(l, 2, groups=2, top_groups=1)[0].tolist() == [[1, 0]]
    assert R.route(l, 2, groups=2, top_groups=1, group_best=2)[0].tolist() == [[2, 3]]


def test_route_masks():
    inf = np.inf
    ids, w = R.route([[-inf, 0.0, -inf, -inf], [-inf] * 4], 2)
    assert ids.tolist() == [[1, 0], [0, 1]] and w.tolist() == [[1.0, 0.0], [0.0, 0.0]]
    ids, w = R.route([[-inf, -3.0, -inf, -inf]], 2, sigmoid=True, bias=[9.0, 0.0, 0.0, 0.0])
    assert ids.tolist() == [[1, 0]] and w.tolist() == [[1.0, 0.0]]
