"""GPU tests of operands of more than 2^32 bytes: rows at both sides of 2^31 and 2^32 are what they are by themselves."""

import pytest
import torch

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module")
def q():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import block_wise_bit_adam8bit_amd as q
    torch.cuda.set_device(0)
    yield q
    torch.cuda.empty_cache()


def fill(rows, cols, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.empty(rows, cols, dtype=BF16, device="cuda")
    for i in range(0, rows, 10000):
        x[i:i + 10000] = torch.randn(min(10000, rows - i), cols, generator=g, device="cuda")
    return x


def test_layer_norm(q):
    rows, dim = 140000, 16384  # 4.6 GB
    x = fill(rows, dim, 0)
    w, b = (torch.randn(dim, device="cuda") for _ in range(2))
    y, mean, rstd = q.qopt_layer_norm_forward(x, w, b)
    at = torch.tensor([0, 1, 65535, 65536, 131071, 131072, rows - 1], device="cuda")
    assert torch.equal(y[at], q.qopt_layer_norm_forward(x[at], w, b)[0])
    dx, dw, db = q.qopt_layer_norm_backward(x, w, mean, rstd, y)
    assert torch.equal(dx[at], q.qopt_layer_norm_backward(x[at], w, mean[at], rstd[at], y[at])[0])
    del dx
    sums, size = torch.zeros(dim, dtype=torch.float64, device="cuda"), torch.zeros(dim, dtype=torch.float64, device="cuda")
    for i in range(0, rows, 10000):
        part = y[i:i + 10000].double()
        sums += part.sum(0)
        size += part.abs().sum(0)
    # a workgroup's rows, then the 256 groups by sixteens
    assert ((db.double() - sums).abs() <= (rows // 256 + 1 + 32) * 2.0 ** -24 * size).all()


def test_4bit_matrices(q):
    n, k = 150000, 65536  # codes of 4.9 GB
    w = fill(n, k, 1)
    wq = q.qopt_fp4_quantize(w)
    at = torch.tensor([0, 17, 65535, 65536, 131071, 131072, 139000, n - 17, n - 1], device="cuda")
    part = q.qopt_fp4_quantize(w[at].contiguous())
    del w
    assert torch.equal(wq.codes[at], part.codes) and torch.equal(wq.scales[:, at], part.scales[:, :len(at)])
    assert torch.equal(q.qopt_fp4_dequantize(*wq, k, BF16)[at], q.qopt_fp4_dequantize(*part, k, BF16))
    values = q.qopt_fp4_dequantize(*part, k).double()
    for m in (1, 20, 40, 300):
        x = torch.randn(m, k, generator=torch.Generator().manual_seed(m)).to("cuda", BF16)
        xv = q.qopt_fp4_dequantize(*q.qopt_fp4_quantize(x), k).double()
        want, size = xv @ values.t().contiguous(), xv.abs() @ values.abs().t().contiguous()
        got = q.qopt_fp4_linear(x, *wq, F32)[:, at].double()
        assert ((got - want).abs() <= (k + 2) * 2.0 ** -24 * size).all()
        got = q.qopt_fp4_matmul(*wq, *q.qopt_fp4_quantize(x), F32)[at].double()
        assert ((got - want.t()).abs() <= (k + 2) * 2.0 ** -24 * size.t()).all()
