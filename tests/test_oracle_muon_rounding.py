"""Pins of the bound that bfloat16 results of the orthogonalisation are tested with: it holds for stored values of
22 bits, and not for 11 or 13."""

import numpy as np
import pytest
import torch

from oracle import muon


@pytest.mark.parametrize("kind", ["normal", "steep", "spike"])
@pytest.mark.parametrize("rows,cols", [(64, 64), (65, 130), (300, 99)])
def test_fewer_bits_are_seen(rows, cols, kind):
    rng = np.random.default_rng(rows + cols)
    u = rng.normal(size=(rows, cols)) * 1e-3
    if kind == "steep":
        u = u * 0.05 + rng.normal(size=(rows, 3)) @ rng.normal(size=(3, cols)) * 2e-3
    if kind == "spike":
        u[rows // 2, cols // 3] = 1.0
    want, most = muon.result_bound(u)
    off = lambda bits: np.linalg.norm(muon.beyond_half(muon.to_bf16(muon.rounded(u, bits=bits)), want))  # noqa: E731
    assert off(22) <= most / 8
    assert off(13) > 2 * most and off(11) > 16 * most


def test_roundings_to_bf16():
    rng = np.random.default_rng(0)
    x = rng.normal(size=2000) * 10.0 ** rng.integers(-6, 6, 2000)
    x[:4] = 0.0, 1.0, 1.0 + 2.0 ** -8, 255.5 / 256  # between two numbers: to the even one
    y = torch.from_numpy(x).bfloat16().double().numpy()
    assert np.array_equal(muon.to_bf16(x), y)
    assert not muon.beyond_half(y, x).any()
    assert muon.beyond_half(np.array([1.0, 0.0]), np.array([1.0 + 3 * 2.0 ** -8, 0.25])).tolist() == [2.0 ** -7, 0.25]


def grouped(s, steps):
    """Singular values by the grouped way's polynomials, in Python's numbers."""
    a, b, c = muon.COEFFICIENTS
    done = 0
    while done < steps:
        g, q = s * s, 1.0
        for _ in range(min(3, steps - done)):
            p = a + b * g + c * g * g
            q, g = p * q, p * g * p
        s, done = q * s, done + min(3, steps - done)
    return s


@pytest.mark.parametrize("rows,cols", [(1, 1), (4, 9), (9, 4), (6, 6), (40, 70)])
@pytest.mark.parametrize("steps", [1, 2, 3, 4, 5, 7, 9])
def test_the_grouped_way_is_the_same_polynomial(rows, cols, steps):
    """With 52 bits it differs from the definition by rounding alone: 2^-52 in each of at most 10 products per iteration, grown
    by 1 / s of the smallest singular value s on its way to 1 (over 0.02 here): 90 * 50 * 2^-52 = 1e-12 for nine."""
    u = np.random.default_rng(rows * 10 + cols).normal(size=(rows, cols))
    want = muon.newton_schulz(u, steps)
    assert np.abs(muon.rounded(u, steps, bits=52) - want).max() < 1e-11
    left, s, right = np.linalg.svd(u, full_matrices=False)
    assert np.abs(left @ np.diag(grouped(s / np.linalg.norm(s), steps)) @ right - want).max() < 1e-11
