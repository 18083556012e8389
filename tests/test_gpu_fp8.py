"""GPU tests of the 8-bit floating point quantizer and products against the oracle.

Quantization is compared bit for bit.  Products are compared with binary64 in two ways:

* on small integers, whose products and sums are exact in every path, the result is the
  exact sum rounded once;
* on real-valued data within bounds.  Binary32 results: k + 2 roundings of the sum of
  magnitudes, 2^-24 each.  bf16 results of the 8-bit instructions: one rounding, 2^-8 of
  the result, and for each block of 128 its 128 products cut at 2^-17 of the largest, which
  is at most the product of the two block maxima.
"""

import threading

import numpy as np
import pytest
import torch

from oracle import fp8

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


def say(msg):
    print(msg, flush=True)


@pytest.fixture(scope="module")
def q():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import block_wise_bit_adam8bit_amd as q
    torch.cuda.set_device(0)
    return q


def host(t):
    """A tensor's values in binary64, or its code bytes."""
    if t.dtype == torch.float8_e4m3fn:
        t = t.view(torch.uint8)
    return t.detach().cpu().numpy() if t.dtype == torch.uint8 else t.detach().double().cpu().numpy()


def pair(m):
    """Codes and scales as the oracle lays them out: [rows, blocks] or [tile rows, blocks]."""
    codes, scales = host(m.codes), host(m.scales)
    rows, kb = codes.shape[0], codes.shape[1] // 128
    by_rows = scales.shape == (kb, -(-rows // 16) * 16)
    return codes, scales.T[:rows] if by_rows else scales


def reals(rng, rows, cols, dtype):
    """Normal values of sizes that vary from row to row, with a few large columns."""
    x = rng.normal(0, 1, (rows, cols)) * 10.0 ** rng.uniform(-2, 2, (rows, 1))
    if cols:
        x[:, rng.integers(0, cols, 1 + cols // 100)] *= 30
    return torch.from_numpy(x.astype(np.float32)).to("cuda", dtype)


def integers(rng, rows, cols, dtype, most=4):
    return torch.from_numpy(rng.integers(-most, most + 1, (rows, cols)).astype(np.float32)).to("cuda", dtype)


def rounded(x, dtype):
    return host(torch.from_numpy(np.asarray(x)).float().to(dtype))


def same_codes(got, want, what):
    nan = (want[0] & 127) == 127
    assert np.array_equal((got[0] & 127) == 127, nan), what
    assert np.array_equal(got[0][~nan], want[0][~nan]), what
    assert np.array_equal(got[1], want[1]), what


def bound(a, b, dtype, exact_sums):
    """(product in binary64, tolerance) of two quantized matrices for a result of ``dtype``."""
    with np.errstate(all="ignore"):
        want, size = fp8.matmul(a, b)
    half = {F32: 2.0 ** -24, BF16: 2.0 ** -8}[dtype]
    tol = half * np.abs(want) + (a[0].shape[1] + 2) * 2.0 ** -24 * size
    if not exact_sums:
        peak = lambda m: np.abs(fp8.dequantize(*m)).reshape(m[0].shape[0], -1, 128).max(2)  # noqa: E731
        tol += 128 * 2.0 ** -17 * (peak(a) @ peak(b).T)
    return want, tol


# ------------------------------------------------------------------ quantizer

SHAPES = [(1, 1), (1, 128), (127, 129), (128, 128), (300, 515), (2, 1000), (1000, 3), (256, 384)]


@pytest.mark.parametrize("tiles", [False, True])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_quantize(q, rows, cols, dtype, tiles):
    say(f"quantize {rows}x{cols} {dtype} tiles {tiles}")
    x = reals(np.random.default_rng(rows + cols), rows, cols, dtype)
    a, t = q.qopt_fp8_quantize(x, tiles=tiles, transposed=True)
    same_codes(pair(a), fp8.quantize(host(x), tiles), "matrix")
    same_codes(pair(t), fp8.quantize(host(x).T, tiles), "transpose")
    for alone, both in ((q.qopt_fp8_quantize(x, tiles=tiles), a),
                        (q.qopt_fp8_quantize(x, tiles=tiles, normal=False, transposed=True), t)):
        same_codes(pair(alone), pair(both), "one output alone")


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_quantize_strided_rows(q, dtype):
    """Rows apart, and starting where wide loads would be misaligned."""
    rng = np.random.default_rng(4)
    for off, wide in ((0, 520), (1, 301), (8, 320), (3, 512)):
        buf = reals(rng, 130, wide, dtype)
        x = buf[:, off:off + 290]
        a, t = q.qopt_fp8_quantize(x, transposed=True)
        same_codes(pair(a), fp8.quantize(host(x)), f"offset {off}")
        same_codes(pair(t), fp8.quantize(host(x).T), f"offset {off}")


@pytest.mark.parametrize("tiles", [False, True])
def test_quantize_special_values(q, tiles):
    f = np.finfo(np.float32)
    row = np.zeros((9, 130), np.float32)
    row[1, :6] = [np.nan, np.inf, -np.inf, 1.0, -448.0, 3.0]
    row[2] = np.nan
    row[3, 5] = f.max
    row[4, 5:8] = [f.tiny, -f.tiny / 2, 1e-45]
    row[5, :4] = [448.0, np.nextafter(np.float32(448), np.float32(999)), -0.0, 2.0 ** -9]
    row[6, :4] = [448.0, 464.0, 2.0 ** -10, 1.5 * 2.0 ** -9]
    row[7, 0] = 1e-45
    row[8, :3] = [np.inf, 1e30, 1e-30]
    for rows in ([r] for r in range(9)) if not tiles else (list(range(9)), [3], [4], [7]):
        x = torch.from_numpy(row[rows]).cuda()
        a, t = q.qopt_fp8_quantize(x, tiles=tiles, transposed=True)
        same_codes(pair(a), fp8.quantize(row[rows], tiles), f"rows {rows}")
        same_codes(pair(t), fp8.quantize(row[rows].T, tiles), f"rows {rows}, transposed")


def test_quantize_rounds_every_midpoint(q):
    """Every border between two codes, its neighbours in binary32, at several scales."""
    mags = fp8.decode_table()[:127]
    mid = ((mags[:-1] + mags[1:]) / 2).astype(np.float32)
    v = np.concatenate([mid, np.nextafter(mid, np.float32(0)), np.nextafter(mid, np.float32(999)), mags])
    rows = []
    for e in (-100, -3, 0, 40, 110):
        b = np.zeros((-(-v.size // 127), 128), np.float32)
        b[:, 0] = 448
        b[:, 1:].reshape(-1)[:0] = 0
        flat = np.resize(np.concatenate([v, -v]), (b.shape[0], 127))
        b[:, 1:] = flat
        rows.append(b * np.float32(2.0 ** e))
    x = np.concatenate(rows)
    same_codes(pair(q.qopt_fp8_quantize(torch.from_numpy(x).cuda())), fp8.quantize(x), "midpoints")


# ------------------------------------------------------------------ products

# one tile, ragged tiles, products that split k (long, few tiles), and ones of big tiles (the last
# three: enough tiles of 256 x 256 to be worth it)
MNK = [(1, 1, 1), (33, 31, 129), (128, 128, 128), (129, 257, 300), (40, 1000, 520), (300, 200, 4096),
       (513, 260, 640), (256, 512, 1152), (700, 36, 96), (65, 130, 9000), (2300, 7000, 130),
       (4096, 4096, 256), (4000, 4100, 640)]


@pytest.mark.parametrize("tiles", [False, True])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("m,n,k", MNK)
def test_matmul(q, m, n, k, dtype, tiles):
    say(f"matmul {m}x{n}x{k} {dtype} tiles {tiles}")
    rng = np.random.default_rng(m + n + k)
    a = q.qopt_fp8_quantize(integers(rng, m, k, F32))
    b = q.qopt_fp8_quantize(integers(rng, n, k, F32), tiles=tiles)
    got = host(q.qopt_fp8_matmul(*a, *b, dtype))
    assert np.array_equal(got, rounded(fp8.matmul(pair(a), pair(b))[0], dtype)), "integers"
    a = q.qopt_fp8_quantize(reals(rng, m, k, F32))
    b = q.qopt_fp8_quantize(reals(rng, n, k, F32), tiles=tiles)
    got = q.qopt_fp8_matmul(*a, *b, dtype)
    want, tol = bound(pair(a), pair(b), dtype, dtype == F32)
    err = np.abs(host(got) - want)
    assert np.all(err <= tol), f"{err.max()} {(err / tol).max()}"
    assert torch.equal(got, q.qopt_fp8_matmul(*a, *b, dtype)), "a second call"


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("m,n", [(130, 200), (2048, 4096), (3000, 3100)])
def test_every_number_of_blocks(q, m, n, dtype):
    """One to nine blocks along the sum: fewer, as many and more than the steps that a kernel
    has under way, in tiles of each size."""
    for kb in range(1, 10):
        rng = np.random.default_rng(kb)
        k = kb * 128 - (kb % 3)
        x, w = integers(rng, m, k, F32), integers(rng, n, k, F32)
        want = (x.double() @ w.double().T).to(dtype)
        a = q.qopt_fp8_quantize(x)
        for tiles in (False, True):
            got = q.qopt_fp8_matmul(*a, *q.qopt_fp8_quantize(w, tiles=tiles), dtype)
            assert torch.equal(got, want), (k, tiles)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_matmul_into_strided_rows(q, dtype):
    """Rows of the result apart and at odd offsets; what lies between them stays."""
    rng = np.random.default_rng(9)
    m, n, k = 150, 270, 256
    a, b = (q.qopt_fp8_quantize(integers(rng, r, k, F32)) for r in (m, n))
    want = q.qopt_fp8_matmul(*a, *b, dtype)
    for off, wide in ((0, 280), (1, 273), (8, 512), (4, 276)):
        buf = torch.full((m, wide), 77, dtype=dtype, device="cuda")
        q.qopt_fp8_matmul(*a, *b, dtype, out=buf[:, off:off + n])
        assert torch.equal(buf[:, off:off + n], want)
        assert bool((buf[:, :off] == 77).all()) and bool((buf[:, off + n:] == 77).all())


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_nan_stays_in_its_row_and_column(q, dtype):
    rng = np.random.default_rng(11)
    m, n, k = 70, 300, 400
    x, w = integers(rng, m, k, F32), integers(rng, n, k, F32)
    x[5, 77], x[9, 300], w[200, 13] = float("nan"), float("inf"), float("-inf")
    got = host(q.qopt_fp8_matmul(*q.qopt_fp8_quantize(x), *q.qopt_fp8_quantize(w, tiles=True), dtype))
    want = np.zeros((m, n), bool)
    want[[5, 9]], want[:, 200] = True, True
    assert np.array_equal(np.isnan(got), want)
    few = host(q.qopt_fp8_linear(x[:10], *q.qopt_fp8_quantize(w, tiles=True), dtype))
    assert np.array_equal(np.isnan(few), want[:10])


@pytest.mark.parametrize("m", [5, 150])
@pytest.mark.parametrize("x_size,w_size", [(1e37, 1e-37), (1e-36, 1e36), (1e-38, 1e38), (1e-41, 1e38),
                                           (1e38, 1e-38), (1e-20, 1e-18), (1e-19, 1e-25)])
def test_sizes_at_the_ends_of_the_range(q, x_size, w_size, m):
    """Scales near both ends: as everywhere, but that binary32 results may take element values
    under 2^-126 as 0, and that a subnormal result is off by half a step of its own (2^-150 and
    2^-134) besides, and each binary32 sum before it by 2^-150."""
    rng = np.random.default_rng(1)
    x = torch.from_numpy(np.clip(rng.normal(0, 1, (m, 260)), -2.5, 2.5) * x_size).float().cuda()
    w = torch.from_numpy(np.clip(rng.normal(0, 1, (70, 260)), -2.5, 2.5) * w_size).float().cuda()
    a, b = q.qopt_fp8_quantize(x), q.qopt_fp8_quantize(w, tiles=True)
    for dtype in (F32, BF16):
        want, tol = bound(pair(a), pair(b), dtype, dtype == F32)
        tol += (2.0 ** -134 if dtype == BF16 else 0) + 400 * 2.0 ** -150
        if dtype == F32:
            va, vb = (np.abs(fp8.dequantize(*pair(t))) for t in (a, b))
            tol += np.where(va < 2.0 ** -126, va, 0) @ vb.T + va @ np.where(vb < 2.0 ** -126, vb, 0).T
        for got in (q.qopt_fp8_matmul(*a, *b, dtype), q.qopt_fp8_linear(x, *b, dtype)):
            err = np.abs(host(got) - want)
            assert np.all(err <= tol), (dtype, err.max(), (err / tol).max())


def test_out_that_overlaps_is_refused(q):
    x = torch.ones(40, 128, device="cuda")
    w = q.qopt_fp8_quantize(torch.ones(128, 128, device="cuda"), tiles=True)
    with pytest.raises(ValueError):
        q.qopt_fp8_linear(x, *w, out=x)
    a = q.qopt_fp8_quantize(x)
    room = torch.empty(40 * 128 * 4, dtype=torch.uint8, device="cuda")
    codes = room[100 * 16:100 * 16 + 40 * 128].view(torch.float8_e4m3fn).view(40, 128)
    codes.copy_(a.codes)
    with pytest.raises(ValueError):
        q.qopt_fp8_matmul(codes, a.scales, *w, F32, out=room.view(F32).view(40, 128))
    got = q.qopt_fp8_matmul(codes, a.scales, *w, F32, out=torch.empty(40, 128, device="cuda"))
    assert bool((got == 128).all())


@pytest.mark.parametrize("m", [3, 80])
def test_without_gradients(q, m):
    """No gradient wanted: the result of the quantized weight, whatever the leaves ask for."""
    x = torch.randn(m, 300, device="cuda", dtype=BF16, requires_grad=True)
    w = torch.randn(70, 300, device="cuda", requires_grad=True)
    want = q.qopt_fp8_linear(x.detach(), *q.qopt_fp8_quantize(w.detach(), tiles=True))
    with torch.no_grad():
        y = q.fp8_linear(x, w)
    assert not y.requires_grad and torch.equal(y, want)
    assert torch.equal(q.fp8_linear(x.detach().view(1, m, 300), w.detach())[0], want)
    wide = torch.zeros(m, 310, device="cuda", dtype=BF16)
    wide[:, 5:305] = x.detach()
    assert torch.equal(q.fp8_linear(wide[:, 5:305], w.detach()), want)
    assert torch.equal(q.fp8_linear(x.detach().t().contiguous().t(), w.detach()), want)
    same = q.fp8_linear(x.detach()[:1].expand(m, 300), w.detach())
    assert torch.equal(same, want[:1].expand(m, 70))


def test_empty_products(q):
    z = lambda r, k: q.Fp8Matrix(torch.empty(r, k, dtype=torch.float8_e4m3fn, device="cuda"),  # noqa: E731
                                 torch.empty(k // 128, -(-r // 16) * 16, dtype=torch.uint8, device="cuda"))
    assert q.qopt_fp8_matmul(*z(0, 128), *z(5, 128)).shape == (0, 5)
    assert q.qopt_fp8_matmul(*z(5, 128), *z(0, 128)).shape == (5, 0)
    for dtype in (F32, BF16):
        out = torch.full((5, 9), 7.0, device="cuda", dtype=dtype)
        q.qopt_fp8_matmul(*z(5, 0), *z(7, 0), dtype, out=out[:, :7])
        assert bool((out[:, :7] == 0).all()) and bool((out[:, 7:] == 7).all())
        assert bool((q.qopt_fp8_linear(torch.empty(3, 0, device="cuda"), *z(7, 0), dtype) == 0).all())
    assert q.qopt_fp8_linear(torch.empty(2, 0, 100, device="cuda"), *z(7, 128)).shape == (2, 0, 7)
    x = torch.empty(0, 100, device="cuda", requires_grad=True)
    w = torch.ones(7, 100, device="cuda", requires_grad=True)
    y = q.fp8_linear(x, w)
    dx, dw = torch.autograd.grad(y, (x, w), torch.empty_like(y))
    assert dx.shape == (0, 100) and dw.shape == (7, 100) and not dw.any()
    for n, k in ((0, 100), (7, 0)):
        x = torch.ones(3, k, device="cuda", requires_grad=True)
        w = torch.ones(n, k, device="cuda", requires_grad=True)
        y = q.fp8_linear(x, w)
        dx, dw = torch.autograd.grad(y, (x, w), torch.ones_like(y))
        assert y.shape == (3, n) and not y.any() and not dx.any() and dw.shape == (n, k)


# ------------------------------------------------------------------ linear

@pytest.mark.parametrize("out_dtype", [F32, BF16])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("m", [1, 2, 15, 16, 17, 32, 33, 100])
def test_linear(q, m, dtype, out_dtype):
    for n, k in ((1, 1), (17, 130), (160, 1024), (500, 2600)):
        say(f"linear {m} rows {n}x{k} {dtype} -> {out_dtype}")
        rng = np.random.default_rng(m + n + k)
        for tiles in (True, False):
            w = q.qopt_fp8_quantize(integers(rng, n, k, F32), tiles=tiles)
            x = integers(rng, m, k, dtype)
            xq = fp8.quantize(host(x))
            got = host(q.qopt_fp8_linear(x, *w, out_dtype))
            assert np.array_equal(got, rounded(fp8.matmul(xq, pair(w))[0], out_dtype)), "integers"
            w = q.qopt_fp8_quantize(reals(rng, n, k, F32), tiles=tiles)
            x = reals(rng, m, k, dtype)
            got = host(q.qopt_fp8_linear(x, *w, out_dtype))
            want, tol = bound(fp8.quantize(host(x)), pair(w), out_dtype, out_dtype == F32)
            assert np.all(np.abs(got - want) <= tol)


@pytest.mark.parametrize("m", [3, 20, 70])
def test_linear_strides_and_shapes(q, m):
    rng = np.random.default_rng(5)
    n, k = 300, 516
    w = q.qopt_fp8_quantize(integers(rng, n, k, F32), tiles=True)
    x = integers(rng, m, k, BF16)
    want = q.qopt_fp8_linear(x, *w)
    for off, wide in ((0, 520), (1, 517), (3, 640)):
        buf = torch.full((m, wide), float("nan"), dtype=BF16, device="cuda")
        buf[:, off:off + k] = x
        out = torch.full((m, n + 5), 77, dtype=BF16, device="cuda")
        q.qopt_fp8_linear(buf[:, off:off + k], *w, out=out[:, 2:2 + n])
        assert torch.equal(out[:, 2:2 + n], want)
        assert bool((out[:, :2] == 77).all()) and bool((out[:, 2 + n:] == 77).all())
    assert torch.equal(q.qopt_fp8_linear(x.view(1, m, k), *w)[0], want)
    assert torch.equal(q.qopt_fp8_linear(x[0], *w), want[0]) or m > 32
    # a token's result does not depend on how many others come with it, up to the few rows' limit
    if m <= 32:
        assert torch.equal(q.qopt_fp8_linear(x[:1], *w), want[:1])


def test_past_32_bit_offsets(q):
    """Weights of more than 2^32 code bytes and results past 2^31 elements."""
    k, n = 4096, (1 << 20) + 40000
    say(f"weights {n}x{k}")
    g = torch.Generator(device="cuda").manual_seed(1)
    codes = torch.randint(0, 4, (n, k), dtype=torch.uint8, device="cuda", generator=g).mul_(8).add_(0x30)
    codes = codes.view(torch.float8_e4m3fn)
    scales = torch.randint(118, 122, (k // 128, n), dtype=torch.uint8, device="cuda", generator=g)
    spots = [0, 1000, (1 << 20) - 1, 1 << 20, n - 1]
    part = (host(codes[spots]), host(scales[:, spots].t()))
    rng = np.random.default_rng(2)
    for m in (2, 2100):
        x = integers(rng, m, k, BF16, 2)
        out = q.qopt_fp8_linear(x, codes, scales)
        want = rounded(fp8.matmul(fp8.quantize(host(x[-2:])), part)[0], BF16)
        assert np.array_equal(host(out[-2:, spots]), want)
        del out


# ------------------------------------------------------------------ gradients

@pytest.mark.parametrize("wdt", [F32, BF16])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("m,n,k", [(1, 1, 1), (5, 130, 70), (130, 300, 257), (600, 128, 520)])
def test_gradients_follow_the_formula(q, m, n, k, dtype, wdt):
    say(f"gradients {m}x{n}x{k} {dtype} weight {wdt}")
    rng = np.random.default_rng(m * n + k)
    x = reals(rng, m, k, dtype).requires_grad_()
    w = reals(rng, n, k, wdt).requires_grad_()
    dy = reals(rng, m, n, dtype)
    y = q.fp8_linear(x, w)
    dx, dw = torch.autograd.grad(y, (x, w), dy)
    assert (y.dtype, dx.dtype, dw.dtype) == (dtype, dtype, wdt)
    X, W, D = host(x), host(w), host(dy)
    for got, a, b, dt in ((y, fp8.quantize(X), fp8.quantize(W, True), dtype),
                          (dx, fp8.quantize(D), fp8.quantize(W.T, True), dtype),
                          (dw, fp8.quantize(D.T), fp8.quantize(X.T), wdt)):
        want, tol = bound(a, b, dt, dt == F32)
        assert np.all(np.abs(host(got) - want) <= tol)
    # one gradient alone is the same one
    assert torch.equal(torch.autograd.grad(q.fp8_linear(x, w.detach()), x, dy)[0], dx)
    assert torch.equal(torch.autograd.grad(q.fp8_linear(x.detach(), w), w, dy)[0], dw)


def test_gradients_are_differences(q):
    """On integers, whose quantization is exact, the layer is the linear map itself, so that
    central differences with a step of 1 equal the gradients exactly."""
    rng = np.random.default_rng(8)
    m, n, k = 3, 5, 140
    x, w, dy = integers(rng, m, k, F32, 3), integers(rng, n, k, F32, 3), integers(rng, m, n, F32, 3)
    loss = lambda a, b: float((q.fp8_linear(a, b).double() * dy.double()).sum())  # noqa: E731
    xr, wr = x.clone().requires_grad_(), w.clone().requires_grad_()
    dx, dw = torch.autograd.grad(q.fp8_linear(xr, wr), (xr, wr), dy)
    for t, grad, at in ((x, dx, [(0, 0), (1, 77), (2, 139)]), (w, dw, [(0, 0), (4, 128), (2, 139)])):
        for i in at:
            v = float(t[i])
            t[i] = v + 1
            up = loss(x, w)
            t[i] = v - 1
            down = loss(x, w)
            t[i] = v
            assert (up - down) / 2 == float(grad[i])


def test_broadcast_and_shared_leaves(q):
    """A broadcast input's gradient is the sum over its copies, a weight used twice gets
    both gradients, leading dimensions and strides are free."""
    rng = np.random.default_rng(3)
    w = integers(rng, 40, 40, F32, 2).requires_grad_()
    x = integers(rng, 1, 40, F32, 2).requires_grad_()
    y = q.fp8_linear(x.expand(6, 40).view(2, 3, 40), w)
    dy = integers(rng, 6, 40, F32, 2).view(2, 3, 40)
    dx, dw = torch.autograd.grad(y, (x, w), dy)
    assert torch.equal(dx, (dy.view(6, 40) @ w).sum(0, keepdim=True).detach())
    assert torch.equal(dw, (dy.view(6, 40).t() @ x.expand(6, 40)).detach())
    a = integers(rng, 40, 8, F32, 2).t().requires_grad_()   # rows not contiguous
    s = q.fp8_linear(a, w) + q.fp8_linear(a, w.t())
    d = integers(rng, 8, 40, F32, 2)
    da, dw = torch.autograd.grad(s, (a, w), d)
    assert torch.equal(da, (d @ w + d @ w.t()).detach())
    assert torch.equal(dw, (d.t() @ a + a.t() @ d).detach())
    y = q.fp8_linear(x, w).sum()
    (g,) = torch.autograd.grad(y, x, create_graph=True)
    with pytest.raises(RuntimeError):  # the backward pass has no derivative of its own
        g.sum().backward()


# ------------------------------------------------------------------ streams, graphs, threads

def test_runs_on_the_callers_stream(q):
    rng = np.random.default_rng(6)
    x, w = integers(rng, 200, 600, BF16), integers(rng, 300, 600, BF16)
    wq = q.qopt_fp8_quantize(w, tiles=True)
    want, few = q.qopt_fp8_linear(x, *wq), q.qopt_fp8_linear(x[:4], *wq)
    big = torch.randn(4096, 4096, device="cuda")
    late = torch.zeros_like(x)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        for _ in range(6):
            big = big @ big * 1e-2
        late.copy_(x)
        got, got_few = q.qopt_fp8_linear(late, *wq), q.qopt_fp8_linear(late[:4], *wq)
    side.synchronize()
    assert torch.equal(got, want) and torch.equal(got_few, few)


def test_captured_calls_replay(q):
    """Forward and backward captured into a graph and replayed on new inputs, with the
    program's eager work between the replays."""
    rng = np.random.default_rng(7)
    x = integers(rng, 300, 400, BF16).requires_grad_()
    w = integers(rng, 500, 400, F32).requires_grad_()
    dy = integers(rng, 300, 500, BF16)

    def step():
        y = q.fp8_linear(x, w)
        dx, dw = torch.autograd.grad(y, (x, w), dy)
        return y.detach(), dx, dw, q.qopt_fp8_linear(x.detach()[:3], *q.qopt_fp8_quantize(w.detach(), tiles=True))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = step()
    for r in range(4):
        with torch.no_grad():
            x.copy_(integers(rng, 300, 400, BF16)), w.copy_(integers(rng, 500, 400, F32))
            dy.copy_(integers(rng, 300, 500, BF16))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(kept, step()):
            assert torch.equal(a, b), f"replay {r}"


def test_two_threads(q):
    rng = np.random.default_rng(12)
    jobs = [(integers(rng, 300, 700, BF16), q.qopt_fp8_quantize(integers(rng, 400, 700, F32), tiles=True))
            for _ in range(2)]
    want = [q.qopt_fp8_linear(x, *w) for x, w in jobs]
    got = [None, None]
    torch.cuda.synchronize()

    def work(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(20):
                got[i] = q.qopt_fp8_linear(jobs[i][0], *jobs[i][1])
            torch.cuda.current_stream().synchronize()

    ts = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    [t.start() for t in ts], [t.join() for t in ts]
    for a, b in zip(got, want):
        assert torch.equal(a, b)


# ------------------------------------------------------------------ the operators together

def test_training_step_in_8_bits(q):
    """Embedding, two linear layers and AdamW, as a training program uses them: every
    parameter moves, the packed weights serve the trained layer, and a second run from the
    same start gives the same bits (nothing here depends on the order of atomics)."""
    def run():
        emb = q.StableEmbedding(64, 256, dtype=BF16, seed=1)
        up, down = q.Fp8Linear(256, 512, seed=2), q.Fp8Linear(512, 64, dtype=BF16, seed=3)
        params = [*emb.parameters(), *up.parameters(), *down.parameters()]
        opt = q.AdamW(params, lr=1e-2, weight_decay=0.1)
        before = [p.detach().clone() for p in params]
        g = torch.Generator(device="cuda").manual_seed(5)
        ids = torch.randint(0, 64, (4, 33), device="cuda", generator=g)
        for _ in range(3):
            opt.zero_grad()
            h = torch.nn.functional.silu(up(emb(ids)))
            loss = torch.nn.functional.cross_entropy(down(h).float().view(-1, 64), ids.view(-1))
            loss.backward()
            norm = torch.stack([p.grad.float().norm() for p in params]).norm()
            opt.step(grad_scale=(1.0 / norm.clamp(min=1.0)).float().view(1))
        assert all(bool(torch.isfinite(p).all()) for p in params)
        assert all(not torch.equal(a, b.detach()) for a, b in zip(before, params))
        kinds = [("m_codes" in opt.state[p]) for p in params]
        assert kinds == [p.numel() >= 4096 for p in params]
        x = emb(ids)[0].detach()
        with torch.no_grad():
            y = up(x)
        assert torch.equal(q.qopt_fp8_linear(x, *up.pack()), y)
        return params

    for a, b in zip(run(), run()):
        assert torch.equal(a, b)


# ------------------------------------------------------------------ every instance of the kernels

def blocks_of_integers(gen, rows, cols, tiles=False):
    """Small integers, times 1, 2 or 4 from block to block of 128 (or tile): their sums of products
    over up to 2^12 columns are exact in binary32, and scales that are taken from another block show."""
    kb = -(-cols // 128)
    x = torch.randint(-4, 5, (rows, kb * 128), device="cuda", generator=gen).float()
    size = torch.randint(0, 3, (-(-rows // 128) if tiles else rows, kb), device="cuda", generator=gen)
    if tiles:
        size = size.repeat_interleave(128, 0)[:rows]
    return (x.view(rows, kb, 128) * (2.0 ** size).unsqueeze(2)).view(rows, kb * 128)[:, :cols].contiguous()


def by_blocks(v, scales):
    """[rows, columns] of codes' values times their scales, in binary64 on the GPU."""
    rows, kb = v.shape[0], v.shape[1] // 128
    e = scales.double() - 127
    e = e[:, :rows].t() if e.shape == (kb, -(-rows // 16) * 16) else e.repeat_interleave(128, 0)[:rows]
    return (v.view(rows, kb, 128) * (2.0 ** e).unsqueeze(2)).view(rows, kb * 128)


def values(matrix):
    """What a quantized matrix stands for."""
    return by_blocks(matrix.codes.double(), matrix.scales)


def peaks(matrix):
    """The largest magnitude of every 8 places of a row, codes under 2^-6 taken as 2^-6."""
    v = by_blocks(matrix.codes.double().abs().clamp(min=2.0 ** -6), matrix.scales)
    return v.view(v.shape[0], -1, 8).amax(2)


def within(got, a, b, dtype):
    """Whether a product of quantized matrices is right: one rounding, k + 2 roundings of the sum of
    magnitudes in binary32, and for bf16, where the 8-bit instructions cut 7 of 8 products at 2^-13 of
    the largest one's power of two, that of every 8 places."""
    av, bv = values(a), values(b)
    want, half = av @ bv.t(), {F32: 2.0 ** -24, BF16: 2.0 ** -8}[dtype]
    tol = half * want.abs() + (av.shape[1] + 2) * 2.0 ** -24 * (av.abs() @ bv.abs().t())
    if dtype == BF16:
        tol += 7 * 2.0 ** -13 * (peaks(a) @ peaks(b).t())
    return bool(((got.double() - want).abs() <= tol).all())


@pytest.mark.parametrize("tiles", [False, True])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("m,n", [(4093, 4090), (4349, 16891)])
def test_every_number_of_blocks_in_large_tiles(q, m, n, dtype, tiles):
    """One to nine blocks along the sum in tiles of 256 x 256: one round of whole tiles, and four rounds
    with the last one's tiles in halves; ragged on every side, into rows that lie apart."""
    gen = torch.Generator(device="cuda").manual_seed(m)
    for kb in range(1, 10):
        k = kb * 128 - (kb % 3)
        say(f"{m}x{n}x{k} {dtype} tiles {tiles}")
        x, w = blocks_of_integers(gen, m, k), blocks_of_integers(gen, n, k, tiles)
        out = torch.full((m, n + 3), 77, dtype=dtype, device="cuda")
        q.qopt_fp8_matmul(*q.qopt_fp8_quantize(x), *q.qopt_fp8_quantize(w, tiles=tiles), dtype, out=out[:, 1:n + 1])
        assert torch.equal(out[:, 1:n + 1], (x.double() @ w.double().t()).to(dtype))
        assert bool((out[:, 0] == 77).all()) and bool((out[:, n + 1:] == 77).all())


def few_rows_runs(n, m, size):
    """Runs of 16 weight rows that a workgroup takes for few rows of x: the library's rule, restated."""
    cost = lambda r: -(-(-(-n // (16 * r))) // 256) * (16 * r + m * size)  # noqa: E731
    return min(range(1, 5), key=cost)


FEW_N, FEW_M = (300, 4113, 8209, 12289, 50257), (1, 16, 17, 32)


def test_the_few_rows_cases_take_every_instance():
    for dtype in (4, 2):
        for ms in ((1, 16), (17, 32)):  # one and two fragments of 16 rows
            assert {few_rows_runs(n, m, dtype) for n in FEW_N for m in ms} == {1, 2, 3, 4}


@pytest.mark.parametrize("tiles", [False, True])
@pytest.mark.parametrize("out_dtype", [F32, BF16])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("n", FEW_N)
def test_few_rows_of_x(q, n, dtype, out_dtype, tiles):
    """Every number of runs and fragments, with weight rows, rows of x and columns that end inside a
    workgroup's; exact sums, and reals within the bounds."""
    gen = torch.Generator(device="cuda").manual_seed(n)
    rng = np.random.default_rng(n)
    for k in (130, 1156):
        w = blocks_of_integers(gen, n, k, tiles)
        wq = q.qopt_fp8_quantize(w, tiles=tiles)
        r = q.qopt_fp8_quantize(reals(rng, n, k, F32), tiles=tiles)
        for m in FEW_M:
            say(f"{m} rows, {n}x{k} {dtype} -> {out_dtype} tiles {tiles}")
            x = blocks_of_integers(gen, m, k).to(dtype)
            out = torch.full((m, n + 3), 77, dtype=out_dtype, device="cuda")
            q.qopt_fp8_linear(x, *wq, out_dtype, out=out[:, 1:n + 1])
            assert torch.equal(out[:, 1:n + 1], (x.double() @ w.double().t()).to(out_dtype))
            assert bool((out[:, 0] == 77).all()) and bool((out[:, n + 1:] == 77).all())
            x = reals(rng, m, k, dtype)
            got = q.qopt_fp8_linear(x, *r, out_dtype)
            assert within(got, q.qopt_fp8_quantize(x), r, out_dtype)


@pytest.mark.parametrize("grad_mode", [False, True])
@pytest.mark.parametrize("m", [3, 80])
def test_a_traced_layer(q, m, grad_mode):
    layer = q.Fp8Linear(300, 70, dtype=BF16, seed=4)
    x, other = (torch.randn(r, 300, device="cuda", dtype=BF16) for r in (m, m + 40))
    with torch.set_grad_enabled(grad_mode):
        traced = torch.jit.trace(layer, (x,))
        for t in (x, other):
            assert torch.equal(traced(t), layer(t))
    got, want = (torch.autograd.grad(f(other).float().square().sum(), layer.weight)[0] for f in (traced, layer))
    assert torch.equal(got, want)


@pytest.mark.parametrize("m", [3, 40])
@pytest.mark.parametrize("k", [128, 384])
def test_products_that_cancel(q, k, m):
    """Two products of 2^16 that cancel beside k - 2 of 2^-j.  The 8-bit instructions cut what is small
    next to the largest of 8 products, so bf16 results are bounded by the operands and not by the
    result; binary32 results are exact while all sums, of at most 2^17 in steps of 2^-j, fit 24 bits."""
    for j in range(10):
        x = torch.full((m, k), 2.0 ** -j, device="cuda")
        w = torch.ones(70, k, device="cuda")
        x[:, :2], w[:, 0], w[:, 1] = 256, 256, -256
        wq = q.qopt_fp8_quantize(w, tiles=True)
        got = {dtype: q.qopt_fp8_linear(x, *wq, dtype) for dtype in (F32, BF16)}
        xq = q.qopt_fp8_quantize(x)
        want = values(xq) @ values(wq).t()
        say(f"2^-{j}: {float(want[0, 0])} as bf16 {float(got[BF16][0, 0])}, as fp32 {float(got[F32][0, 0])}")
        for dtype, y in got.items():
            assert within(y, xq, wq, dtype)
        if j <= 6:
            assert torch.equal(got[F32].double(), want)


@pytest.mark.parametrize("at", [0, 40, 64, 120])
@pytest.mark.parametrize("least,most", [(0, 127), (0, 20), (100, 127)])
def test_what_8_bit_products_lose(q, at, least, most):
    """Eight places of codes of every size, of which two products cancel exactly, so that the other six
    are all that is left: 200 x 3000 combinations within the bound."""
    gen = torch.Generator(device="cuda").manual_seed(at + most)

    def matrix(rows):
        codes = torch.zeros(rows, 128, dtype=torch.uint8, device="cuda")
        codes[:, at:at + 8] = torch.randint(least, most, (rows, 8), device="cuda", generator=gen) \
            + 128 * torch.randint(0, 2, (rows, 8), device="cuda", generator=gen)
        codes[:, at + 1] = codes[:, at]
        return codes

    a, b = matrix(200), matrix(3000)
    b[:, at + 1] ^= 128
    a, b = (q.Fp8Matrix(c.view(torch.float8_e4m3fn),
                        torch.randint(120, 135, (1, -(-len(c) // 16) * 16), dtype=torch.uint8, device="cuda", generator=gen))
            for c in (a, b))
    for dtype in (BF16, F32):
        assert within(q.qopt_fp8_matmul(*a, *b, dtype), a, b, dtype)


@pytest.mark.parametrize("m", [3, 40])
def test_the_largest_magnitudes(q, m):
    """From 1.9375 * 2^127 on a value rounds to 2^128, which counts as infinity where the result is
    binary32 and is multiplied as it is where it is bf16; one under that is ordinary in both."""
    x = torch.ones(m, 256, device="cuda")
    x[0], x[1] = 0, 0
    x[0, 3], x[1, 200] = 3.39e38, 3.28e38  # 2^128 and 240 * 2^120
    w = torch.full((70, 256), 2.0 ** -20, device="cuda")
    w[5] = 0
    wq = q.qopt_fp8_quantize(w, tiles=True)
    want = values(q.qopt_fp8_quantize(x)) @ values(wq).t()
    assert float(want[0, 0]) == 2.0 ** 108 and float(want[1, 0]) == 240 * 2.0 ** 100
    assert torch.equal(q.qopt_fp8_linear(x, *wq, BF16).double(), want)
    exact = q.qopt_fp8_linear(x, *wq, F32)
    assert torch.equal(exact[1:].double(), want[1:])
    assert not bool(torch.isfinite(exact[0]).any())
