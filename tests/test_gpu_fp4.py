"""GPU tests of the 4-bit quantizer and products against the oracle.

Quantization is compared bit for bit.  Products are compared with binary64 in two ways:

* on small integers, whose products and sums are exact, the result is the exact sum rounded once;
* on real-valued data within k + 2 binary32 roundings of the sum of magnitudes, 2^-24 each (the products
  themselves are exact), and half a step of the result.
"""

import threading

import numpy as np
import pytest
import torch

from oracle import fp4, fp8

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
HALF = {F32: 2.0 ** -24, BF16: 2.0 ** -8}


def say(msg):
    print(msg, flush=True)


@pytest.fixture(scope="module")
def q():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import block_wise_bit_adam8bit_amd as q
    torch.cuda.set_device(0)
    return q


def host(t):
    return t.detach().cpu().numpy() if t.dtype == torch.uint8 else t.detach().double().cpu().numpy()


def pair(m):
    return fp4.unpack(host(m.codes), host(m.scales))


def reals(rng, rows, cols, dtype):
    """Normal values of sizes that vary from row to row, with a few large columns."""
    x = rng.normal(0, 1, (rows, cols)) * 10.0 ** rng.uniform(-2, 2, (rows, 1))
    if cols:
        x[:, rng.integers(0, cols, 1 + cols // 100)] *= 30
    return torch.from_numpy(x.astype(np.float32)).to("cuda", dtype)


def integers(rng, rows, cols, dtype):
    """Integers that 4-bit blocks hold as they are: 4 and 6 are the largest codes at a scale of 1."""
    return torch.from_numpy(rng.choice([-6, -4, -3, -2, -1, 0, 1, 2, 3, 4, 6], (rows, cols)).astype(np.float32)).to("cuda", dtype)


def same_matrix(got, want):
    codes, scales = fp4.pack(*want)
    assert np.array_equal(host(got.scales), scales)
    assert np.array_equal(host(got.codes), codes)


def bound(a, b, dtype):
    with np.errstate(all="ignore"):
        want, size = fp4.matmul(a, b)
    return want, HALF[dtype] * np.abs(want) + (a[0].shape[1] + 2) * 2.0 ** -24 * size


# ------------------------------------------------------------------ quantizer

SHAPES = [(1, 1), (1, 32), (17, 33), (16, 256), (127, 129), (300, 515), (2, 1000), (1000, 3), (33, 513), (5, 2051)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_quantize_and_dequantize(q, rows, cols, dtype):
    say(f"quantize {rows}x{cols} {dtype}")
    x = reals(np.random.default_rng(rows + cols), rows, cols, dtype)
    m = q.qopt_fp4_quantize(x)
    want = fp4.quantize(host(x))
    same_matrix(m, want)
    values = fp4.dequantize(*want)[:, :cols]
    for out in (F32, BF16):  # two significant bits: exact in both
        assert np.array_equal(host(q.qopt_fp4_dequantize(*m, cols, out)), values)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_strided_rows(q, dtype):
    """Rows apart, and starting where wide accesses would be misaligned."""
    rng = np.random.default_rng(4)
    for off, wide in ((0, 620), (1, 601), (8, 640), (3, 999)):
        buf = reals(rng, 35, wide, dtype)
        x = buf[:, off:off + 590]
        m = q.qopt_fp4_quantize(x)
        same_matrix(m, fp4.quantize(host(x)))
        out = torch.full((35, wide), 77, dtype=dtype, device="cuda")
        q.qopt_fp4_dequantize(*m, 590, dtype, out=out[:, off:off + 590])
        assert torch.equal(out[:, off:off + 590], q.qopt_fp4_dequantize(*m, 590, dtype))
        assert bool((out[:, :off] == 77).all()) and bool((out[:, off + 590:] == 77).all())


def test_special_values(q):
    f = np.finfo(np.float32)
    x = np.zeros((9, 70), np.float32)
    x[1, :6] = [np.nan, 2.0, 1.0, 1.0, -448.0, 3.0]
    x[2, 40] = -np.inf
    x[3, 5] = f.max
    x[4, 5:8] = [f.tiny, -f.tiny / 2, 1e-45]
    x[5, :4] = [6.0, np.nextafter(np.float32(6), np.float32(999)), -0.0, 0.25]
    x[6, :4] = [6.0, 5.0, -0.25, 0.75]
    x[7, 0] = 1e-45
    x[8, :3] = [3e38, 1e30, 1e-30]
    for dtype in (F32, BF16):
        t = torch.from_numpy(x).to("cuda", dtype)
        m = q.qopt_fp4_quantize(t)
        want = fp4.quantize(host(t))
        same_matrix(m, want)
        with np.errstate(over="ignore"):
            values = torch.from_numpy(fp4.dequantize(*want)[:, :70]).float()
        for out in (F32, BF16):  # through binary32, as the kernel: its subnormals are exact here
            assert torch.equal(q.qopt_fp4_dequantize(*m, 70, out).cpu().nan_to_num(1234.0), values.to(out).nan_to_num(1234.0))


def test_every_midpoint(q):
    """Every border between two codes, its neighbours in binary32, at several scales."""
    mags = fp4.decode_table()[:8]
    mid = ((mags[:-1] + mags[1:]) / 2).astype(np.float32)
    v = np.concatenate([mid, np.nextafter(mid, np.float32(0)), np.nextafter(mid, np.float32(999)), mags])
    flat = np.resize(np.concatenate([v, -v]), (31, 31)).astype(np.float32)
    b = np.concatenate([np.full((31, 1), 6, np.float32), flat], 1)
    x = np.concatenate([b * np.float32(2.0 ** e) for e in (-120, -3, 0, 40, 125)])
    same_matrix(q.qopt_fp4_quantize(torch.from_numpy(x).cuda()), fp4.quantize(x))


def test_every_bf16_of_a_block(q):
    """All finite bf16 values next to a largest one of each size."""
    bits = torch.arange(0, 1 << 16, dtype=torch.int32).to(torch.int16).view(BF16)
    v = bits[bits.isfinite()].float()
    v = v[v.abs() < 2.0 ** 100]
    v = torch.nn.functional.pad(v, (0, -v.numel() % 31)).view(-1, 31)
    v = torch.cat([v.abs().amax(1, keepdim=True) * 1.25, v], 1).to(BF16)
    same_matrix(q.qopt_fp4_quantize(v.cuda()), fp4.quantize(host(v)))


# ------------------------------------------------------------------ products

# one tile, ragged tiles, products that split k (long, few tiles), and ones of big tiles (the last four)
MNK = [(1, 1, 1), (33, 31, 129), (128, 128, 256), (129, 257, 300), (40, 1000, 520), (300, 200, 4096),
       (513, 260, 640), (256, 512, 1152), (700, 36, 96), (65, 130, 20000), (2300, 7000, 130),
       (4096, 4096, 256), (4000, 4100, 1340), (2049, 9000, 600)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("m,n,k", MNK)
def test_matmul(q, m, n, k, dtype):
    say(f"matmul {m}x{n}x{k} {dtype}")
    rng = np.random.default_rng(m + n + k)
    x, w = integers(rng, m, k, F32), integers(rng, n, k, F32)
    a, b = q.qopt_fp4_quantize(x), q.qopt_fp4_quantize(w)
    got = q.qopt_fp4_matmul(*a, *b, dtype)
    assert torch.equal(got, (x.double() @ w.double().t().contiguous()).to(dtype)), "integers"
    a, b = (q.qopt_fp4_quantize(reals(rng, r, k, F32)) for r in (m, n))
    got = q.qopt_fp4_matmul(*a, *b, dtype)
    want, tol = bound(pair(a), pair(b), dtype)
    err = np.abs(host(got) - want)
    assert np.all(err <= tol), f"{err.max()} {(err / tol).max()}"
    assert torch.equal(got, q.qopt_fp4_matmul(*a, *b, dtype)), "a second call"


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("m,n", [(130, 200), (2048, 4096), (3000, 3100)])
def test_every_number_of_steps(q, m, n, dtype):
    """One to nine steps along the sum: fewer, as many and more than a kernel has under way, in tiles of each size."""
    for steps in range(1, 10):
        rng = np.random.default_rng(steps)
        k = steps * 256 - (steps % 3) * 70
        x, w = integers(rng, m, k, F32), integers(rng, n, k, F32)
        got = q.qopt_fp4_matmul(*q.qopt_fp4_quantize(x), *q.qopt_fp4_quantize(w), dtype)
        assert torch.equal(got, (x.double() @ w.double().t().contiguous()).to(dtype)), k


def test_blocks_of_different_scales(q):
    """Powers of two that differ from block to block and row to row: exact sums show a scale in the wrong place."""
    rng = np.random.default_rng(3)
    for m, n, k in ((40, 70, 1100), (300, 300, 700), (2100, 4200, 520)):
        # products between 2^-4 and 2^12, sums below 2^23 of the smallest step
        x, w = (integers(rng, r, k, F32) * torch.from_numpy(2.0 ** rng.integers(-2, 3, (r, -(-k // 32))))
                .float().cuda().repeat_interleave(32, 1)[:, :k] for r in (m, n))
        a, b = q.qopt_fp4_quantize(x), q.qopt_fp4_quantize(w)
        va, vb = q.qopt_fp4_dequantize(*a, k).double(), q.qopt_fp4_dequantize(*b, k).double()
        want = (va @ vb.t().contiguous()).float()
        assert torch.equal(q.qopt_fp4_matmul(*a, *b, F32), want)
        assert torch.equal(q.qopt_fp4_linear(x, *b), want)
        assert torch.equal(q.qopt_fp4_linear(x[:7], *b), want[:7])


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_matmul_into_strided_rows(q, dtype):
    rng = np.random.default_rng(9)
    for m, n, k in ((150, 270, 256), (3, 270, 300)):
        x = integers(rng, m, k, F32)
        a, b = q.qopt_fp4_quantize(x), q.qopt_fp4_quantize(integers(rng, n, k, F32))
        want = q.qopt_fp4_matmul(*a, *b, dtype)
        for off, wide in ((0, 280), (1, 273), (8, 512), (4, 276)):
            for call in (lambda o: q.qopt_fp4_matmul(*a, *b, dtype, out=o), lambda o: q.qopt_fp4_linear(x, *b, dtype, out=o)):
                buf = torch.full((m, wide), 77, dtype=dtype, device="cuda")
                call(buf[:, off:off + n])
                assert torch.equal(buf[:, off:off + n], want)
                assert bool((buf[:, :off] == 77).all()) and bool((buf[:, off + n:] == 77).all())


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_nan_stays_in_its_row_and_column(q, dtype):
    rng = np.random.default_rng(11)
    m, n, k = 70, 300, 600
    x, w = integers(rng, m, k, F32), integers(rng, n, k, F32)
    x[5, 77], x[9, 590], w[200, 13], w[299, 300] = float("nan"), float("inf"), float("-inf"), float("nan")
    wq = q.qopt_fp4_quantize(w)
    got = host(q.qopt_fp4_matmul(*q.qopt_fp4_quantize(x), *wq, dtype))
    want = np.zeros((m, n), bool)
    want[[5, 9]], want[:, [200, 299]] = True, True
    assert np.array_equal(np.isnan(got), want)
    few = host(q.qopt_fp4_linear(x[:10], *wq, dtype))
    assert np.array_equal(np.isnan(few), want[:10])
    fine = ~want
    clean = host(q.qopt_fp4_matmul(*q.qopt_fp4_quantize(x.nan_to_num(0, 0, 0)), *q.qopt_fp4_quantize(w.nan_to_num(0, 0, 0)), dtype))
    assert np.array_equal(got[fine], clean[fine]) and np.array_equal(few[fine[:10]], clean[:10][fine[:10]])


@pytest.mark.parametrize("m", [5, 150])
@pytest.mark.parametrize("x_size,w_size", [(1e37, 1e-37), (1e-36, 1e36), (1e-38, 1e38), (1e-41, 1e38), (1e38, 1e-38),
                                           (1e-20, 1e-18), (1e-19, 1e-25)])
def test_sizes_at_the_ends_of_the_range(q, x_size, w_size, m):
    """Scales near both ends: as everywhere, but that products under 2^-126 may count as 0, a subnormal
    result is off by half a step of its own (2^-150 and 2^-134) and each sum before it by 2^-150."""
    rng = np.random.default_rng(1)
    x = torch.from_numpy(np.clip(rng.normal(0, 1, (m, 260)), -2.5, 2.5) * x_size).float().cuda()
    w = torch.from_numpy(np.clip(rng.normal(0, 1, (70, 260)), -2.5, 2.5) * w_size).float().cuda()
    a, b = q.qopt_fp4_quantize(x), q.qopt_fp4_quantize(w)
    for dtype in (F32, BF16):
        want, tol = bound(pair(a), pair(b), dtype)
        va, vb = (np.abs(fp4.dequantize(*pair(t))) for t in (a, b))
        small = np.zeros_like(want)
        for l in range(260):
            p = va[:, l:l + 1] * vb[:, l]
            small += np.where(p < 2.0 ** -126, p, 0)
        tol += small + (2.0 ** -134 if dtype == BF16 else 0) + 400 * 2.0 ** -150
        for got in (q.qopt_fp4_matmul(*a, *b, dtype), q.qopt_fp4_linear(x, *b, dtype)):
            err = np.abs(host(got) - want)
            assert np.all(err <= tol), (dtype, err.max(), (err / tol).max())


@pytest.mark.parametrize("x_dtype,out", [(BF16, BF16), (F32, F32), (BF16, F32), (F32, BF16)])
@pytest.mark.parametrize("m", [1, 2, 15, 16, 17, 31, 32, 33, 130])
def test_linear(q, m, x_dtype, out):
    """Few rows in one launch and more in two, for widths of each number of weight rows per workgroup."""
    for n, k in ((1, 1), (5, 33), (16, 256), (70, 300), (500, 2048), (4096, 511), (9000, 520), (13000, 257), (17000, 70), (30000, 300)):
        rng = np.random.default_rng(m + n + k)
        x, w = integers(rng, m, k, x_dtype), q.qopt_fp4_quantize(integers(rng, n, k, BF16))
        got = q.qopt_fp4_linear(x, *w, out)
        wv = q.qopt_fp4_dequantize(*w, k).double()
        assert torch.equal(got, (x.double() @ wv.t().contiguous()).to(out)), (n, k)
        x = reals(rng, m, k, x_dtype)
        got = q.qopt_fp4_linear(x, *w, out)
        want, tol = bound(fp4.quantize(host(x)), pair(w), out)
        err = np.abs(host(got) - want)
        assert np.all(err <= tol), (n, k, (err / tol).max())
        assert torch.equal(got, q.qopt_fp4_linear(x, *w, out))


def test_a_row_does_not_depend_on_the_others(q):
    rng = np.random.default_rng(17)
    w = q.qopt_fp4_quantize(reals(rng, 300, 700, BF16))
    x = reals(rng, 32, 700, BF16)
    whole = q.qopt_fp4_linear(x, *w)
    for m in (1, 5, 16, 17):
        assert torch.equal(q.qopt_fp4_linear(x[:m], *w), whole[:m])
    assert torch.equal(q.qopt_fp4_linear(x.view(2, 16, 700), *w), whole.view(2, 16, 300))


def test_out_that_overlaps_is_refused(q):
    x = torch.ones(40, 256, device="cuda")
    w = q.qopt_fp4_quantize(torch.ones(256, 256, device="cuda"))
    with pytest.raises(ValueError):
        q.qopt_fp4_linear(x, *w, out=x)
    a = q.qopt_fp4_quantize(x)
    room = torch.zeros(5120 + 4 * 40 * 256, dtype=torch.uint8, device="cuda")
    codes = room[:5120].view(40, 128)
    codes.copy_(a.codes)
    with pytest.raises(ValueError):
        q.qopt_fp4_dequantize(codes, a.scales, 256, F32, out=room[4096:4096 + 4 * 40 * 256].view(F32).view(40, 256))
    assert bool((q.qopt_fp4_dequantize(codes, a.scales, 256, F32, out=room[5120:].view(F32).view(40, 256)) == 1).all())
    buf = torch.zeros(40, 512, device="cuda")
    buf[:, :256] = x
    q.qopt_fp4_linear(buf[:, :256], *w, out=buf[:, 256:])
    assert bool((buf[:, 256:] == 256).all()) and bool((buf[:, :256] == 1).all())
    with pytest.raises(ValueError):
        q.qopt_fp4_linear(buf[:, :256], *w, out=buf[:, 255:511])


def test_empty_products(q):
    z = lambda r, k: q.Fp4Matrix(torch.empty(r, k // 2, dtype=torch.uint8, device="cuda"),  # noqa: E731
                                 torch.empty(k // 128, -(-r // 16) * 16, 4, dtype=torch.uint8, device="cuda"))
    assert q.qopt_fp4_matmul(*z(0, 256), *z(5, 256)).shape == (0, 5)
    assert q.qopt_fp4_matmul(*z(5, 256), *z(0, 256)).shape == (5, 0)
    assert q.qopt_fp4_dequantize(*z(0, 256), 200).shape == (0, 200)
    assert q.qopt_fp4_dequantize(*z(3, 0), 0).shape == (3, 0)
    assert q.qopt_fp4_quantize(torch.empty(3, 0, device="cuda")).codes.shape == (3, 0)
    for dtype in (F32, BF16):
        out = torch.full((5, 9), 7.0, device="cuda", dtype=dtype)
        q.qopt_fp4_matmul(*z(5, 0), *z(7, 0), dtype, out=out[:, :7])
        assert bool((out[:, :7] == 0).all()) and bool((out[:, 7:] == 7).all())
        assert bool((q.qopt_fp4_linear(torch.empty(3, 0, device="cuda"), *z(7, 0), dtype) == 0).all())
    assert q.qopt_fp4_linear(torch.empty(2, 0, 100, device="cuda"), *z(7, 256)).shape == (2, 0, 7)
    for m, n, k in ((0, 7, 100), (3, 0, 100), (3, 7, 0)):
        x = torch.ones(m, k, device="cuda", requires_grad=True)
        w = torch.ones(n, k, device="cuda", requires_grad=True)
        y = q.fp4_linear(x, w)
        dx, dw = torch.autograd.grad(y, (x, w), torch.ones_like(y))
        assert y.shape == (m, n) and not y.any() and dx.shape == (m, k) and dw.shape == (n, k)
        assert not dx.any() and not dw.any()


# ------------------------------------------------------------------ the layer

def layer_data(m, n, k, act, weight, seed=0):
    rng = np.random.default_rng(seed + m + n + k)
    x, dy = reals(rng, m, k, act), (reals(rng, m, n, F32) * 1e-3).to(act)
    return x, reals(rng, n, k, weight), dy


def eight(x, tiles=False):
    return fp8.dequantize(*fp8.quantize(host(x) if torch.is_tensor(x) else x, tiles))


def gradient_bounds(x, w, dy, act, weight):
    """(value, most it may be off) of dx and dw: products over 8-bit codes.  bf16 results cut each of a
    block's 128 products at 2^-17 of the largest; binary32 ones round their sums."""
    out = []
    for a, b, dtype in ((eight(dy), eight(host(w).T, True), act), (eight(host(dy).T), eight(host(x).T), weight)):
        want, size = a @ b.T, abs(a) @ abs(b).T
        tol = HALF[dtype] * abs(want) + (a.shape[1] + 2) * 2.0 ** -24 * size
        if dtype == BF16:
            peak = lambda v: abs(v).reshape(v.shape[0], -1, 128).max(2)  # noqa: E731
            tol += 128 * 2.0 ** -17 * (peak(a) @ peak(b).T)
        out.append((want, tol))
    return out


@pytest.mark.parametrize("act,weight", [(BF16, F32), (BF16, BF16), (F32, F32), (F32, BF16)])
@pytest.mark.parametrize("m,n,k", [(1, 5, 7), (20, 70, 300), (33, 128, 256), (200, 130, 520), (600, 300, 129)])
def test_layer_and_gradients(q, m, n, k, act, weight):
    x, w, dy = layer_data(m, n, k, act, weight)
    x, w = x.requires_grad_(), w.requires_grad_()
    y = q.fp4_linear(x, w)
    dx, dw = torch.autograd.grad(y, (x, w), dy)
    assert y.dtype == dx.dtype == act and dw.dtype == weight
    # the forward pass is what a server computes
    assert torch.equal(y, q.qopt_fp4_linear(x.detach(), *q.qopt_fp4_quantize(w.detach())))
    with torch.no_grad():
        assert torch.equal(y, q.fp4_linear(x, w))
    want, tol = bound(fp4.quantize(host(x)), fp4.quantize(host(w)), act)
    assert np.all(abs(host(y) - want) <= tol)
    for t, (want, tol) in zip((dx, dw), gradient_bounds(x, w, dy, act, weight)):
        err = abs(host(t) - want)
        assert np.all(err <= tol), (err / tol).max()
    for leaf, g in ((x, dx), (w, dw)):  # one alone
        x1, w1 = (t.detach().requires_grad_(t is leaf) for t in (x, w))
        assert torch.equal(torch.autograd.grad(q.fp4_linear(x1, w1), x1 if leaf is x else w1, dy)[0], g)


def test_gradients_are_those_of_the_8bit_layer(q):
    x, w, dy = layer_data(70, 200, 300, BF16, F32)
    got, want = [], []
    for layer, to in ((q.fp4_linear, got), (q.fp8_linear, want)):
        x1, w1 = x.detach().requires_grad_(), w.detach().requires_grad_()
        to += torch.autograd.grad(layer(x1, w1), (x1, w1), dy)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_gradients_against_differences(q):
    """Straight through the quantization the layer is linear: with operands that both formats hold as they are,
    differences of the forward pass are its gradients, exactly."""
    rng = np.random.default_rng(8)
    x, w, dy = (integers(rng, r, c, F32) for r, c in ((40, 96), (24, 96), (40, 24)))
    x, w = x.requires_grad_(), w.requires_grad_()
    dx, dw = torch.autograd.grad(q.fp4_linear(x, w), (x, w), dy)
    with torch.no_grad():
        loss = lambda a, b: (q.fp4_linear(a, b).double() * dy.double()).sum()  # noqa: E731
        for _ in range(10):
            d, e = integers(rng, 40, 96, F32), integers(rng, 24, 96, F32)
            # a linear function's differences: of the second operand at the first, and the other way round
            assert (loss(d, w) - loss(torch.zeros_like(d), w)).item() == (dx.double() * d.double()).sum().item()
            assert (loss(x, e) - loss(x, torch.zeros_like(e))).item() == (dw.double() * e.double()).sum().item()


def test_layer_inputs_of_other_shapes(q):
    x, w, dy = layer_data(24, 70, 300, BF16, F32)
    want = q.fp4_linear(x, w)
    for v in (x.view(2, 12, 300), x.t().contiguous().t(), x.repeat(1, 2)[:, :300]):
        v1 = v.detach().requires_grad_()
        w1 = w.t().contiguous().t().requires_grad_()
        y = q.fp4_linear(v1, w1)
        assert torch.equal(y.reshape(24, 70), want)
        dx, dw = torch.autograd.grad(y.sum(), (v1, w1))  # an upstream gradient that is broadcast
        assert dx.shape == v.shape and dw.shape == w.shape
    y = q.fp4_linear(x[0], w)
    assert y.shape == (70,) and torch.equal(y, want[0])
    assert torch.equal(q.fp4_linear(x[:1].expand(24, 300), w), want[:1].expand(24, 70))


def test_the_callers_stream_and_a_captured_pass(q):
    x, w, dy = layer_data(300, 200, 520, BF16, F32, 5)
    x, w = x.requires_grad_(), w.requires_grad_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.autograd.grad(q.fp4_linear(x, w), (x, w), dy)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = q.fp4_linear(x, w)
        got = [y, *torch.autograd.grad(y, (x, w), dy)]
    for i in range(4):
        fx, fw, fdy = layer_data(300, 200, 520, BF16, F32, 50 + i)
        with torch.no_grad():
            x.copy_(fx), w.copy_(fw), dy.copy_(fdy)
        graph.replay()
        torch.cuda.synchronize()
        x1, w1 = fx.requires_grad_(), fw.requires_grad_()
        y1 = q.fp4_linear(x1, w1)
        want = [y1, *torch.autograd.grad(y1, (x1, w1), fdy)]
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_two_threads_at_once(q):
    jobs = []
    for i, m in enumerate((7, 600)):
        rng = np.random.default_rng(30 + i)
        jobs.append((reals(rng, m, 2048, BF16), *q.qopt_fp4_quantize(reals(rng, 700, 2048, BF16))))
    want = [q.qopt_fp4_linear(*j) for j in jobs]
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(20):
                y = q.qopt_fp4_linear(*jobs[i])
                torch.cuda.current_stream().synchronize()
                if not torch.equal(y, want[i]):
                    wrong.append(i)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert not wrong


def test_forward_mode_is_refused_and_a_trace_holds_the_layer(q):
    import torch.autograd.forward_ad as fwd
    x, w, _ = layer_data(5, 64, 96, F32, F32)
    with fwd.dual_level():
        with pytest.raises(NotImplementedError):
            q.fp4_linear(fwd.make_dual(x, torch.ones_like(x)), w)
    m = q.Fp4Linear(96, 64, seed=3)
    traced = torch.jit.trace(m, x, check_trace=False)
    y = x * 2 + 1
    assert torch.equal(traced(y), m(y))
    wq = m.pack()
    assert torch.equal(q.qopt_fp4_linear(y, *wq), m(y))
    with pytest.raises(RuntimeError):
        torch.jit.trace(lambda t: q.qopt_fp4_linear(t, *wq), x, check_trace=False)
    assert "96, 64" in repr(m) and not torch.equal(q.Fp4Linear(96, 64).weight, q.Fp4Linear(96, 64).weight)
