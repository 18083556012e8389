"""Pins of the Newton-Schulz oracle: by singular values, and torch's optimizer for the step."""

import numpy as np
import pytest
import torch

from oracle import muon


def scalar(s, steps):
    a, b, c = muon.COEFFICIENTS
    for _ in range(steps):
        s = a * s + b * s ** 3 + c * s ** 5
    return s


@pytest.mark.parametrize("rows,cols", [(1, 1), (4, 9), (9, 4), (6, 6)])
@pytest.mark.parametrize("steps", [1, 3, 5, 7])
def test_singular_values_move_by_the_polynomial(rows, cols, steps):
    u = np.random.default_rng(rows * 10 + cols).normal(size=(rows, cols))
    left, s, right = np.linalg.svd(u, full_matrices=False)
    want = left @ np.diag(scalar(s / np.linalg.norm(s), steps)) @ right
    assert np.abs(muon.newton_schulz(u, steps) - want).max() < 1e-12
    # the grouped way is the same polynomial: with 52 bits it differs by rounding alone
    assert np.abs(muon.rounded(u, steps) - want).max() < 1e-4
    assert np.abs(muon.rounded(u, steps, bf16=True) - want).max() < 0.05


def test_zero_and_tiny_matrices():
    assert not muon.newton_schulz(np.zeros((3, 4))).any() and not muon.rounded(np.zeros((3, 4))).any()
    u = np.full((1, 1), 1e-9)  # divided by eps, not by its norm
    assert np.allclose(muon.newton_schulz(u), scalar(1e-2, 5))


def test_the_step_is_that_of_torch():
    if not hasattr(torch.optim, "Muon"):
        pytest.skip("this torch has no Muon")
    rng = np.random.default_rng(3)
    for adjust in ("original", "match_rms_adamw"):
        for nesterov in (True, False):
            p0 = rng.normal(size=(6, 4)).astype(np.float32)
            p = torch.nn.Parameter(torch.from_numpy(p0.copy()))
            opt = torch.optim.Muon([p], lr=0.02, momentum=0.9, weight_decay=0.1, nesterov=nesterov, adjust_lr_fn=adjust)
            want, m = p0.astype(np.float64), np.zeros((6, 4), np.float32)
            for _ in range(3):
                g = rng.normal(size=(6, 4)).astype(np.float32)
                p.grad = torch.from_numpy(g)
                opt.step()
                m, u = muon.momentum(g, m, 0.9, nesterov)
                o = muon.newton_schulz(u)
                want = want * muon.decay(0.02, 0.1) - o * muon.rate(0.02, 6, 4, adjust)
            # torch iterates in bf16: 8 bits, ten of them in a step
            assert np.abs(p.detach().numpy() - want).max() < 3 * 0.02 * 1.3 * 0.1
            assert np.abs(opt.state[p]["momentum_buffer"].numpy() - m).max() < 1e-6
