"""The router's oracle on NaN logits, by hand and against rows with -inf in their place."""
import numpy as np

from oracle import int4_ref as R

NAN, INF = np.nan, np.inf


def test_by_hand():
    for bias in (None, [0.0, 0.0, 0.0]):
        ids, w = R.route([[NAN, 1.0, 1.0], [NAN, -INF, NAN]], 3, bias=bias)
        assert ids.tolist() == [[1, 2, 0], [0, 1, 2]] and w.tolist() == [[0.5, 0.5, 0.0], [0.0, 0.0, 0.0]]
    ids, w = R.route([[NAN, 0.0, 0.0]], 2, sigmoid=True, renormalise=False)
    assert ids.tolist() == [[1, 2]] and w.tolist() == [[0.5, 0.5]]


def test_is_a_mask():
    r = np.random.default_rng(0)
    l = r.standard_normal((20, 16))
    l[r.random(l.shape) < 0.4] = -INF
    other = np.where(np.isneginf(l), NAN, l)
    for sigmoid in (False, True):
        for bias in (None, r.standard_normal(16)):
            for best in (1, 2):
                for renormalise in (False, True):
                    kw = dict(sigmoid=sigmoid, bias=bias, groups=4, top_groups=2, group_best=best, renormalise=renormalise)
                    for a, b in zip(R.route(l, 4, **kw), R.route(other, 4, **kw)):
                        assert np.array_equal(a, b)
