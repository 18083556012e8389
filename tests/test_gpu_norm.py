"""GPU tests of layer normalisation against binary64.

Bounds, with u = 2^-24 (one binary32 rounding).  A sum over a row is a chain of at most D additions
(a thread's own values, 6 steps of a wave, its waves), so it is off by D u of the sum of magnitudes.
With that for the mean, half of it for the root of the variance and one u per further operation:
    h  is off by  eh = u (|h| (D / 2 + 8) + D mean|x| rstd)
    y  by  |w| eh + 4 u (|h w| + |b|)
    dx by  rstd (4 u |v| + (D + 4) u mean|v| + |h| (mean(|v| eh) + (D + 6) u mean|v h|) + eh |mean v h|)
           + (D / 2 + 8) u rstd (|v| + |mean v| + |h mean v h|)
    dw by  sum(|dy| eh) + R u sum|dy h|,  db by R u sum|dy|,  R the chain of additions over the rows
and each by half a step of its type.
"""

import threading

import numpy as np
import pytest
import torch

from oracle import norm

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
U = 2.0 ** -24
HALF = {F32: 2.0 ** -24, BF16: 2.0 ** -8}

SIZES = [(1, 1), (3, 2), (1, 16), (3, 7), (5, 512), (4, 513), (7, 1000), (2, 1024), (3, 1025), (9, 2048), (601, 2047),
         (1030, 600), (5, 4096), (3, 4099), (2, 8192), (2, 8200), (3, 16384), (2, 16383), (2, 16391), (3, 20000),
         (2500, 40), (530, 2500), (3, 4104), (600, 5121), (520, 6144), (2, 6145), (300, 9000), (270, 10241), (3, 12288), (2, 12289),
         (3, 24569), (300, 16392), (4, 9), (700, 15), (9, 511), (70, 5), (2049, 8), (300, 1023), (40, 8193)]


@pytest.fixture(scope="module")
def q():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import block_wise_bit_adam8bit_amd as q
    torch.cuda.set_device(0)
    return q


def host(t):
    return t.detach().double().cpu().numpy()


def chain(dim):
    """Additions behind each other in a sum over a row."""
    return (32 if dim <= 16384 else -(-dim // 1024)) + 6 + 16


def row_chain(rows):
    groups = min(rows, 512)
    return -(-rows // max(1, groups)) + 4 + -(-groups // 16) + 16


def data(rows, dim, dtype, wdtype, seed=0):
    g = torch.Generator().manual_seed(seed * 1000003 + rows * 1009 + dim)
    x = torch.randn(rows, dim, generator=g) * 10.0 ** torch.empty(rows, 1).uniform_(-2, 2, generator=g)
    x += torch.randn(rows, 1, generator=g)
    w, b = torch.randn(dim, generator=g), torch.randn(dim, generator=g)
    dy = torch.randn(rows, dim, generator=g) * 0.01
    return x.to(dtype).cuda(), w.to(wdtype).cuda(), b.to(wdtype).cuda(), dy.to(dtype).cuda()


def bounds(x, w, b, dy, dtype, wdtype, eps=1e-5):
    """(values, most that they may be off) of y, dx, dw, db."""
    rows, dim = x.shape
    D, R = chain(dim), row_chain(rows)
    y, h, _, rstd = norm.layer_norm(x, w, b, eps)
    dx, dw, db = norm.layer_norm_backward(x, w, dy, eps)
    w1, b1 = np.ones(dim) if w is None else w, np.zeros(dim) if b is None else b
    v = dy * w1
    mean = lambda a: a.mean(1, keepdims=True)  # noqa: E731
    eh = U * (abs(h) * (D / 2 + 8) + D * mean(abs(x)) * rstd)
    ey = abs(w1) * eh + 4 * U * (abs(h * w1) + abs(b1)) + HALF[dtype] * abs(y)
    s1 = mean(v * h)
    ex = rstd * (4 * U * abs(v) + (D + 4) * U * mean(abs(v))
                 + abs(h) * (mean(abs(v) * eh) + (D + 6) * U * mean(abs(v * h))) + eh * abs(s1)) \
        + (D / 2 + 8) * U * rstd * (abs(v) + abs(mean(v)) + abs(h * s1)) + HALF[dtype] * abs(dx)
    ew = (abs(dy) * eh).sum(0) + R * U * abs(dy * h).sum(0) + HALF[wdtype] * abs(dw)
    eb = R * U * abs(dy).sum(0) + HALF[wdtype] * abs(db)
    return (y, ey), (dx, ex), (dw, ew), (db, eb)


def close(t, value, most, what):
    off = abs(host(t) - value)
    # what rounds to the type's subnormals is off by half of its smallest step
    assert (off <= most + 2.0 ** -134).all(), f"{what}: {(off / (most + 1e-300)).max()} of what it may be off"


@pytest.mark.parametrize("dtype,wdtype", [(BF16, F32), (F32, F32), (BF16, BF16), (F32, BF16)])
@pytest.mark.parametrize("rows,dim", SIZES)
def test_forward_and_gradients(q, rows, dim, dtype, wdtype):
    x, w, b, dy = data(rows, dim, dtype, wdtype)
    want = bounds(host(x), host(w), host(b), host(dy), dtype, wdtype)
    x, w, b = x.requires_grad_(), w.requires_grad_(), b.requires_grad_()
    y = q.layer_norm(x, w, b)
    got = [y, *torch.autograd.grad(y, (x, w, b), dy)]
    for t, like, (value, most), what in zip(got, (x, x, w, b), want, ("y", "dx", "dw", "db")):
        assert t.shape == like.shape and t.dtype == like.dtype
        close(t, value, most, what)
    # the path without gradients and the library calls: the same bits
    with torch.no_grad():
        assert torch.equal(q.layer_norm(x, w, b), y)
        out, mean, rstd = q.qopt_layer_norm_forward(x, w, b)
        assert torch.equal(out, y) and mean.shape == rstd.shape == (rows,)
        again = q.qopt_layer_norm_backward(x, w, mean, rstd, dy)
        assert all(torch.equal(a, c) for a, c in zip(again, got[1:]))


@pytest.mark.parametrize("rows,dim", [(5, 40), (3, 1999), (4, 3000), (2, 9001), (2, 17000)])
def test_without_weight_or_bias(q, rows, dim):
    x, w, b, dy = data(rows, dim, F32, F32, 1)
    for use_w, use_b in ((False, False), (True, False), (False, True)):
        wa, ba = w if use_w else None, b if use_b else None
        hw, hb = host(w) if use_w else None, host(b) if use_b else None
        want = bounds(host(x), hw, hb, host(dy), F32, F32)
        xa = x.clone().requires_grad_()
        leaves = [t.clone().requires_grad_() if t is not None else None for t in (wa, ba)]
        y = q.layer_norm(xa, *leaves)
        given = [xa] + [t for t in leaves if t is not None]
        grads = torch.autograd.grad(y, given, dy)
        which = [0, 1] + ([2] if use_w else []) + ([3] if use_b else [])
        for t, i in zip((y, *grads), which):
            close(t, *want[i], f"output {i}")


def test_only_the_gradients_that_are_wanted(q):
    x, w, b, dy = data(33, 700, BF16, F32, 2)
    _, mean, rstd = q.qopt_layer_norm_forward(x, w, b)
    whole = q.qopt_layer_norm_backward(x, w, mean, rstd, dy)
    for need in ((True, False, False), (False, True, False), (False, False, True), (False, True, True),
                 (False, False, False)):
        part = q.qopt_layer_norm_backward(x, w, mean, rstd, dy, need_x=need[0], need_weight=need[1], need_bias=need[2])
        for a, c, n in zip(part, whole, need):
            assert (a is None) != n and (not n or torch.equal(a, c))


def test_gradients_against_differences(q):
    x, w, b, dy = data(6, 300, F32, F32, 3)
    hx, hw, hb, hdy = (host(t) for t in (x, w, b, dy))
    leaves = [t.clone().requires_grad_() for t in (x, w, b)]
    grads = torch.autograd.grad(q.layer_norm(*leaves), leaves, dy)
    want = bounds(hx, hw, hb, hdy, F32, F32)[1:]
    rng = np.random.default_rng(0)
    loss = lambda *a: (norm.layer_norm(*a)[0] * hdy).sum()  # noqa: E731
    for i, (g, (_, most)) in enumerate(zip(grads, want)):
        at = [hx, hw, hb]
        # steps in proportion to a row's spread: central differences are then off by 1e-10 of the change
        size = np.std(hx, 1, keepdims=True) if i == 0 else 1.0
        d = rng.normal(size=at[i].shape) * size
        t = 1e-5
        hi, lo = ([a + s * t * d if j == i else a for j, a in enumerate(at)] for s in (1, -1))
        off = abs((loss(*hi) - loss(*lo)) / (2 * t) - (host(g) * d).sum())
        assert off <= (most * abs(d)).sum() + 1e-7 * abs(host(g) * d).sum()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("dim", [37, 1024, 3001, 17001])
def test_rows_apart_and_other_columns_left_alone(q, dtype, dim):
    rows = 5
    g = torch.Generator().manual_seed(dim)
    buf = torch.randn(rows, 2 * dim + 3, generator=g).to(dtype).cuda()
    x, out = buf[:, 1:dim + 1], buf[:, dim + 1:2 * dim + 1]
    before = buf.clone()
    want = q.qopt_layer_norm_forward(x.contiguous())[0]
    got, mean, rstd = q.qopt_layer_norm_forward(x, out=out)
    assert got is out and torch.equal(out, want)
    before[:, dim + 1:2 * dim + 1] = want
    assert torch.equal(buf, before)
    dy = torch.randn(rows, dim + 5, generator=g).to(dtype).cuda()[:, 2:dim + 2]
    a = q.qopt_layer_norm_backward(x, None, mean, rstd, dy)
    b = q.qopt_layer_norm_backward(x.contiguous(), None, mean, rstd, dy.contiguous())
    assert all(torch.equal(s, t) for s, t in zip(a, b))
    with pytest.raises(ValueError):
        q.qopt_layer_norm_forward(x, out=buf[:, :dim])


def test_rows_of_one_value_and_constant_rows(q):
    for dim in (1, 64, 5000, 17000):
        x = torch.full((3, dim), 7.0, device="cuda")
        w, b = torch.randn(dim, device="cuda"), torch.randn(dim, device="cuda")
        y, mean, rstd = q.qopt_layer_norm_forward(x, w, b)
        assert torch.equal(y, b.expand(3, dim)) and torch.equal(mean, x[:, 0])
        assert torch.allclose(rstd, torch.full_like(rstd, 1e5 ** 0.5), rtol=4 * U, atol=0)


def test_a_row_that_is_not_finite_leaves_the_others(q):
    for dim in (40, 1000, 3000, 9000, 17001):
        x, w, b, dy = data(9, dim, BF16, F32, 4)
        want = q.qopt_layer_norm_forward(x, w, b)[0]
        y, mean, rstd = q.qopt_layer_norm_forward(x, w, b)
        gx = q.qopt_layer_norm_backward(x, w, mean, rstd, dy)[0]
        bad = x.clone()
        bad[2, dim // 2], bad[5, -1] = float("inf"), float("nan")
        y, mean, rstd = q.qopt_layer_norm_forward(bad, w, b)
        got = q.qopt_layer_norm_backward(bad, w, mean, rstd, dy)
        keep = torch.tensor([i not in (2, 5) for i in range(9)])
        assert torch.equal(y[keep], want[keep]) and torch.equal(got[0][keep], gx[keep])
        assert y[~keep].isnan().all() and got[0][~keep].isnan().all() and got[1].isnan().all()


def test_no_rows_and_no_columns(q):
    for dtype in (F32, BF16):
        w = torch.randn(6, device="cuda", dtype=dtype, requires_grad=True)
        x = torch.empty(2, 0, 6, device="cuda", dtype=dtype, requires_grad=True)
        y = q.layer_norm(x, w, w.detach().clone().requires_grad_())
        gx, gw = torch.autograd.grad(y, (x, w), torch.empty_like(y))
        assert gx.shape == x.shape and torch.equal(gw, torch.zeros_like(w))
        e = torch.empty(3, 0, device="cuda", dtype=dtype, requires_grad=True)
        assert q.layer_norm(e).shape == (3, 0)
        assert torch.autograd.grad(q.layer_norm(e), e, torch.empty_like(e))[0].shape == (3, 0)


def test_inputs_of_other_shapes_and_orders(q):
    x, w, b, dy = data(24, 50, F32, F32, 5)
    want = q.layer_norm(x, w, b)
    assert torch.equal(q.layer_norm(x.view(2, 3, 4, 50), w, b).view(24, 50), want)
    assert torch.equal(q.layer_norm(x[0], w, b), want[0])
    for v in (x.t().contiguous().t(), x.repeat(1, 2)[:, :50], x.view(4, 6, 50).transpose(0, 1).contiguous().transpose(0, 1)):
        v = v.detach().requires_grad_()
        y = q.layer_norm(v, w, b)
        assert torch.equal(y.reshape(24, 50), want)
        g = torch.autograd.grad(y, v, dy.view(y.shape))[0]
        assert g.shape == v.shape
    # an upstream gradient that is broadcast
    x1 = x.clone().requires_grad_()
    ones = torch.autograd.grad(q.layer_norm(x1, w, b), x1, torch.ones_like(x1))[0]
    assert torch.equal(torch.autograd.grad(q.layer_norm(x1, w, b).sum(), x1)[0], ones)


def test_the_callers_stream(q):
    x, w, b, dy = data(4000, 2048, BF16, F32, 6)
    want = q.layer_norm(x, w, b)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        late = x * 0
        for _ in range(20):
            late = late + x * 0.05
        late.copy_(x)
        y = q.layer_norm(late, w, b)
    side.synchronize()
    assert torch.equal(y, want)


def test_a_captured_pass_replayed(q):
    x, w, b, dy = data(700, 1500, BF16, F32, 7)
    x, w, b = x.requires_grad_(), w.requires_grad_(), b.requires_grad_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.autograd.grad(q.layer_norm(x, w, b), (x, w, b), dy)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = q.layer_norm(x, w, b)
        got = [y, *torch.autograd.grad(y, (x, w, b), dy)]
    for i in range(4):
        fresh, _, _, fresh_dy = data(700, 1500, BF16, F32, 8 + i)
        with torch.no_grad():
            x.copy_(fresh)
            dy.copy_(fresh_dy)
        graph.replay()
        torch.cuda.synchronize()
        out, mean, rstd = q.qopt_layer_norm_forward(x.detach(), w.detach(), b.detach())
        want = [out, *q.qopt_layer_norm_backward(x.detach(), w.detach(), mean, rstd, dy)]
        assert all(torch.equal(a, c) for a, c in zip(got, want))


def test_two_threads_at_once(q):
    jobs = [data(900, 1100, BF16, F32, 20 + i) for i in range(2)]
    want = [q.layer_norm(*j[:3]) for j in jobs]
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(20):
                y = q.layer_norm(*jobs[i][:3])
                torch.cuda.current_stream().synchronize()
                if not torch.equal(y, want[i]):
                    wrong.append(i)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert not wrong


def test_forward_mode_is_refused_and_a_trace_holds_the_layer(q):
    import torch.autograd.forward_ad as fwd
    x, w, b, _ = data(5, 64, F32, F32, 9)
    with fwd.dual_level():
        with pytest.raises(NotImplementedError):
            q.layer_norm(fwd.make_dual(x, torch.ones_like(x)), w, b)
    m = q.LayerNorm(64)
    traced = torch.jit.trace(m, x, check_trace=False)
    y, _, _, _ = data(5, 64, F32, F32, 10)
    assert torch.equal(traced(y), m(y))
    with pytest.raises(RuntimeError):
        torch.jit.trace(lambda t: q.qopt_layer_norm_forward(t, w, b)[0], x, check_trace=False)


def test_the_module_trains(q):
    m = q.LayerNorm(48)
    x, _, _, dy = data(10, 48, F32, F32, 11)
    m(x).backward(dy)
    want = bounds(host(x), np.ones(48), np.zeros(48), host(dy), F32, F32)
    close(m.weight.grad, *want[2], "dw")
    close(m.bias.grad, *want[3], "db")
    again = q.LayerNorm(48, bias=False)
    assert again(x).shape == x.shape and "bias=False" in repr(again)
