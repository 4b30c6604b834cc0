"""Pins of the MXFP4 oracle: the format's values, rounding by hand, scales, storage order."""
import numpy as np
import pytest

from oracle import mxfp4_ref as R


def test_e2m1_values():
    assert R.E2M1[:8].tolist() == [0, 0.5, 1, 1.5, 2, 3, 4, 6]
    assert R.E2M1[8:].tolist() == [0, -0.5, -1, -1.5, -2, -3, -4, -6]


def test_e2m1_rounding_by_hand():
    u = np.array([0.25, 0.26, 0.75, 0.74, 1.25, 1.75, 2.5, 2.51, 3.5, 3.49, 5.0, 5.01, 6.9, 7.99, -0.25, -5.0, -0.6])
    want = [0, 1, 2, 1, 2, 4, 4, 5, 6, 5, 6, 7, 7, 7, 8, 14, 9]
    assert R.e2m1_encode(u).tolist() == want


def test_e2m1_round_trip_and_nearest(rng):
    assert R.e2m1_encode(R.E2M1).tolist() == list(range(16))
    u = rng.uniform(-8, 8, 20000)
    got = R.E2M1[R.e2m1_encode(u)]
    best = np.abs(np.clip(u, -6, 6)[:, None] - R.E2M1).min(1)
    assert np.array_equal(np.abs(np.clip(u, -6, 6) - got), best)


@pytest.mark.parametrize("amax,byte", [(4.0, 127), (7.99, 127), (8.0, 128), (1.0, 125), (0.0, 127), (2.0 ** -125, 0),
                                       (2.0 ** -133, 0), (2.0 ** 127, 252), (np.inf, 255), (np.nan, 255)])
def test_scale_bytes(amax, byte):
    v = np.zeros((1, 128))
    v[0, 37] = amax
    assert R.block_scale_bytes(v).tolist() == [[127, byte, 127, 127]]
    codes, s = R.quant(v)
    if byte == 255:
        assert not codes.any() and np.isnan(R.dequant(codes, s)[0, 32:64]).all()


def test_saturation_and_low_bits():
    v = np.zeros((1, 128))
    v[0, :4] = [7.5, 5.0, 0.3, -0.2]          # scale 1: 7.5 saturates to 6, 5 ties to 4
    codes, s = R.quant(v)
    assert R.dequant(codes, s)[0, :4].tolist() == [6, 4, 0.5, 0]
    assert codes[0, :2].tolist() == [7 | 6 << 4, 1 | 8 << 4]


@pytest.mark.parametrize("rows,cols", [(1, 128), (3, 512), (5, 640), (2, 1920)])
def test_storage_order(rows, cols, rng):
    s = rng.integers(0, 256, (rows, cols // 32)).astype(np.uint8)
    st = R.store_scales(s)
    assert np.array_equal(R.load_scales(st, rows, cols), s)
    words = cols // 128
    for r in range(rows):
        for w in range(words):
            at = 4 * rows * (w // 4) + r * min(4, words - 4 * (w // 4)) + w % 4
            assert np.array_equal(st[4 * at:4 * at + 4], s[r, 4 * w:4 * w + 4])


def test_products_and_norm_against_loops(rng):
    x, w = rng.normal(size=(2, 128)), rng.normal(size=(6, 128))
    y, mag = R.gemm_ref(x, w)
    h, _ = R.gated_ref(x, w)
    for i in range(2):
        for j in range(6):
            assert np.isclose(y[i, j], sum(x[i, e] * w[j, e] for e in range(128)), rtol=1e-12)
        for j in range(3):
            g = y[i, j]
            assert np.isclose(h[i, j], g / (1 + np.exp(-g)) * y[i, j + 3], rtol=1e-12)
    assert (mag >= np.abs(y)).all()
    one, two = 0x3F80, 0x4000                  # rows of 2 (1 + 1), weight 2: v = 2 * 2 / sqrt(4 + 5)
    b = np.full((1, 128), one, np.uint16)
    v, t = R.norm_ref(b, b, np.full(128, two, np.uint16), 5.0)
    assert (t == 2).all() and np.allclose(v, 4 / 3)
