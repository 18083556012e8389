"""GPU tests of many Newton-Schulz iterations on matrices of up to 32 rows or columns, which are iterated in binary64.

Rounding of 2^-53 in a direction that the matrix does not have, or hardly, grows by 3.4445 per iteration, as it does in the
definition's own iteration in binary64, until it is one of the matrix's directions: singular values stay under 1.21."""

import numpy as np
import pytest
import torch

from oracle import muon

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
HALF = {F32: 2.0 ** -24, BF16: 2.0 ** -8}
SHAPES = [(2, 3), (20, 50), (50, 20), (32, 32), (32, 300), (1, 40), (7, 2000)]


@pytest.fixture(scope="module")
def q():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import block_wise_bit_adam8bit_amd as q
    torch.cuda.set_device(0)
    return q


def host(t):
    return t.detach().double().cpu().numpy()


def scalar(s, steps):
    a, b, c = muon.COEFFICIENTS
    for _ in range(steps):
        s = a * s + b * s ** 3 + c * s ** 5
    return s


def noise(rows, cols, steps):
    """Sums of up to max(rows, cols) terms in each iteration, 2^-53 each, grown as above, in every one of the places."""
    return 2.0 ** -53 * max(rows, cols) * steps * 3.4445 ** steps * np.sqrt(min(rows, cols))


@pytest.mark.parametrize("steps", [1, 5, 6, 7, 12, 13, 16])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_matrices_of_one_direction(q, rows, cols, steps):
    """Whole numbers, so that there is exactly one."""
    rng = np.random.default_rng(rows + cols)
    left, right = (rng.choice([-3, -2, -1, 1, 2, 3], n).astype(np.float64) for n in (rows, cols))
    want = scalar(1.0, steps) * np.outer(left, right) / (np.linalg.norm(left) * np.linalg.norm(right))
    x = torch.from_numpy(np.outer(left, right).astype(np.float32)).cuda()
    for dtype in (F32, BF16):
        got = host(q.qopt_orthogonalize(x, steps=steps, out_dtype=dtype))
        off = np.linalg.norm(got - want)
        assert off <= HALF[dtype] * np.linalg.norm(want) * 1.01 + noise(rows, cols, steps), (dtype, off)


@pytest.mark.parametrize("steps", [6, 7, 12, 17, 32])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_full_matrices(q, rows, cols, steps):
    """Singular values between 0.5 and 2 of each other: no direction is grown on the way, so that 32 iterations are off by
    rounding alone, of the polynomial whose slope is at most 1.2 near 1 on average (3.4445 through the first two)."""
    rng = np.random.default_rng(steps + rows * cols)
    m = min(rows, cols)
    left, right = (np.linalg.qr(rng.normal(size=(n, m)))[0] for n in (rows, cols))
    s = rng.uniform(1, 2, m)
    x = torch.from_numpy(((left * s) @ right.T).astype(np.float32)).cuda()
    l, s, r = np.linalg.svd(host(x), full_matrices=False)
    want = (l * scalar(s / np.linalg.norm(s), steps)) @ r
    for dtype in (F32, BF16):
        got = host(q.qopt_orthogonalize(x, steps=steps, out_dtype=dtype))
        off = np.linalg.norm(got - want) / np.linalg.norm(want)
        assert off <= HALF[dtype] * 1.01 + 2.0 ** -53 * 300 * 1.2 ** steps * 3.4445 ** 4, (dtype, off)


@pytest.mark.parametrize("rows,cols", SHAPES)
def test_singular_values_stay_bounded(q, rows, cols):
    rng = np.random.default_rng(5)
    one = np.repeat(rng.normal(size=(1, cols)), rows, 0)
    steep = rng.normal(size=(rows, 2)) @ rng.normal(size=(2, cols)) * 1e6 + rng.normal(size=(rows, cols))
    zero = np.zeros((rows, cols))
    zero[rows // 2] = 1.0
    for x in (one, steep, zero):
        for steps in (12, 20, 27, 32):
            got = host(q.qopt_orthogonalize(torch.from_numpy(x.astype(np.float32)).cuda(), steps=steps))
            assert np.isfinite(got).all() and np.linalg.norm(got, 2) <= 1.21


def test_a_step_of_many_iterations(q):
    g = torch.from_numpy(np.outer([1, -2, 3, 1], [2, 1, -1, 3, 1, 1, 2]).astype(np.float32)).cuda()
    p, m = torch.zeros(4, 7, device="cuda"), torch.zeros(4, 7, device="cuda")
    q.qopt_muon32bit_step([(p, g, m)], lr=1.0, momentum=0.0, weight_decay=0.0, nesterov=False, steps=13)
    assert torch.equal(p, -q.qopt_orthogonalize(g, steps=13))
    assert torch.equal(m, g)


@pytest.mark.parametrize("rows,cols", [(33, 40), (100, 300), (300, 99), (700, 900)])
def test_larger_matrices_stay_bounded(q, rows, cols):
    """The same on the way of larger matrices, whose groups begin with A anew; 2^-8 for the destination's own rounding."""
    rng = np.random.default_rng(rows)
    one = np.repeat(rng.normal(size=(1, cols)), rows, 0)
    steep = rng.normal(size=(rows, 2)) @ rng.normal(size=(2, cols)) * 1e6 + rng.normal(size=(rows, cols))
    spread = rng.normal(size=(rows, cols)) * np.exp(3 * rng.normal(size=(rows, 1)))
    for x in (one, steep, spread):
        for steps in (12, 20, 32):
            for dtype in (F32, BF16):
                got = host(q.qopt_orthogonalize(torch.from_numpy(x.astype(np.float32)).cuda(), steps=steps, out_dtype=dtype))
                assert np.isfinite(got).all() and np.linalg.norm(got, 2) <= 1.21 + 2.0 ** -8
