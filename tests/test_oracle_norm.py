"""Pins of the layer normalisation oracle: values by hand, and its gradients by differences."""

import numpy as np

from oracle import norm


def test_values_by_hand():
    y, h, mean, rstd = norm.layer_norm([[1.0, 3.0], [5.0, 5.0]], [2.0, 4.0], [1.0, -1.0], eps=0.0 + 1e-300)
    assert np.array_equal(mean, [[2.0], [5.0]]) and rstd[0, 0] == 1.0
    assert np.array_equal(h[0], [-1.0, 1.0]) and np.array_equal(y[0], [-1.0, 3.0])
    assert np.array_equal(y[1], [1.0, -1.0])  # a constant row leaves the bias


def test_gradients_against_differences():
    rng = np.random.default_rng(5)
    x, w, b, dy = rng.normal(size=(4, 9)), rng.normal(size=9), rng.normal(size=9), rng.normal(size=(4, 9))
    grads = norm.layer_norm_backward(x, w, dy)
    loss = lambda x, w, b: (norm.layer_norm(x, w, b)[0] * dy).sum()  # noqa: E731
    t = 1e-5
    for i, g in enumerate(grads):
        at = [x, w, b]
        d = rng.normal(size=at[i].shape)
        hi, lo = ([a + s * t * d if j == i else a for j, a in enumerate(at)] for s in (1, -1))
        # central differences: an error of t^2 times a third derivative, and 2^-53 |loss| / t
        assert abs((loss(*hi) - loss(*lo)) / (2 * t) - (g * d).sum()) < 1e-7
