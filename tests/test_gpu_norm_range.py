"""GPU tests of layer normalisation where binary32 statistics reach their limits, as the header states them."""

import pytest
import torch

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module")
def q():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import block_wise_bit_adam8bit_amd as q
    torch.cuda.set_device(0)
    return q


@pytest.mark.parametrize("dim", [37, 1000, 2048, 4096, 9001, 16384, 20000])
@pytest.mark.parametrize("away", [1e2, 1e4, 1e6])
def test_rows_far_from_zero(q, dim, away):
    """The mean is off by at most one rounding of 2^-24 for each of the additions behind each other (32 of a thread's own, or
    dim / 1024 in long rows, 6 steps of a wave, 16 waves, the division), and every result by that over the spread; each
    result itself by 8 roundings."""
    x = torch.randn(20, dim, generator=torch.Generator().manual_seed(dim)).cuda() + away
    y, mean, rstd = q.qopt_layer_norm_forward(x)
    d = x.double()
    m = d.mean(1, keepdim=True)
    r = 1 / torch.sqrt((d - m).square().mean(1, keepdim=True) + 1e-5)
    shift = ((32 if dim <= 16384 else -(-dim // 1024)) + 23) * U * m.abs()
    want = (d - m) * r
    assert ((mean.double()[:, None] - m).abs() <= shift).all()
    # a mean that is off by s adds s^2 to the variance
    off = shift * r + want.abs() * ((shift * r).square() / 2 + 64 * U)
    assert ((y.double() - want).abs() <= off).all()


@pytest.mark.parametrize("dim", [40, 3000, 17000])
def test_rows_whose_squares_overflow(q, dim):
    x = torch.randn(4, dim, generator=torch.Generator().manual_seed(dim)).cuda()
    x[1] *= 1e20
    w, b = torch.full((dim,), 2.0, device="cuda"), torch.arange(float(dim), device="cuda")
    y, mean, rstd = q.qopt_layer_norm_forward(x, w, b)
    assert rstd[1].item() == 0 and torch.equal(y[1], b)
    keep = [0, 2, 3]
    assert torch.equal(y[keep], q.qopt_layer_norm_forward(x[keep], w, b)[0])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_rows_without_values(q, dtype):
    """Their mean is that of nothing, as torch's is; nothing that lay in memory before is returned."""
    for shape in ((5, 0), (2, 3, 0), (0, 0), (0, 7)):
        rows = torch.Size(shape[:-1]).numel()
        keep = torch.full((2, rows), 7.0, device="cuda")
        del keep  # the memory that comes next
        x = torch.empty(shape, dtype=dtype, device="cuda", requires_grad=True)
        w, b = (torch.ones(shape[-1], device="cuda", requires_grad=True) for _ in range(2))
        y, mean, rstd = q.qopt_layer_norm_forward(x.detach(), w.detach(), b.detach())
        assert y.shape == shape and mean.shape == rstd.shape == (rows,)
        assert mean.isnan().all() and rstd.isnan().all()
        z = q.layer_norm(x, w, b)
        dx, dw, db = torch.autograd.grad(z, (x, w, b), torch.ones_like(z))
        assert dx.shape == shape and not dw.any() and not db.any() and dw.shape == db.shape == shape[-1:]
