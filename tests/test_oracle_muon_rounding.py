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
