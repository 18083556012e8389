"""GPU tests of the orthogonalisation and the Muon step.

Momentum, its codes and block maxima are compared bit for bit.  An orthogonalised matrix is compared
with the definition in binary64, in the Frobenius norm: 8 times what the oracle's model of the stored
values' rounding moves the same matrix by (its roundings fall otherwise than the kernel's), and as much
again for the binary32 sums of k terms, whose average error of sqrt(k) / 2 roundings of 2^-24 is that many
quarters of a stored value's 2^-22; besides half a step of the destination's type.
"""

import threading

import numpy as np
import pytest
import torch

import oracle
from oracle import muon

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
    return t.detach().double().cpu().numpy()


def gradient(rng, rows, cols, kind="normal"):
    u = rng.normal(size=(rows, cols)) * 1e-3
    if kind == "steep":  # a few directions hold nearly everything
        r = min(3, rows, cols)
        u = u * 0.05 + rng.normal(size=(rows, r)) @ rng.normal(size=(r, cols)) * 2e-3
    return u.astype(np.float32)


def allowance(u, steps, dtype, eps=1e-7):
    """(exact result, how far another may be off it in the Frobenius norm)."""
    want = muon.newton_schulz(u, steps, eps)
    model = np.linalg.norm(muon.rounded(u, steps, eps, dtype == BF16) - want)
    k = max(u.shape)
    return want, 8 * model * (1 + np.sqrt(k) / 8) + 2.0 ** -22 + HALF[dtype] * np.linalg.norm(want)


SHAPES = [(1, 1), (1, 7), (7, 1), (3, 5), (64, 64), (65, 130), (99, 300), (300, 99), (128, 129), (200, 1000), (257, 256),
          (600, 700), (1000, 40), (520, 515)]


@pytest.mark.parametrize("dtype,out", [(F32, F32), (BF16, BF16), (F32, BF16), (BF16, F32)])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_orthogonalize(q, rows, cols, dtype, out):
    say(f"orthogonalize {rows}x{cols} {dtype} {out}")
    rng = np.random.default_rng(rows * 1000 + cols)
    for kind in ("normal", "steep"):
        x = torch.from_numpy(gradient(rng, rows, cols, kind)).to("cuda", dtype)
        got = q.qopt_orthogonalize(x, out_dtype=out)
        assert got.dtype == out and got.shape == x.shape
        want, most = allowance(host(x), 5, out)
        off = np.linalg.norm(host(got) - want)
        assert off <= most, (kind, off, most)
        assert torch.equal(got, q.qopt_orthogonalize(x, out_dtype=out))


@pytest.mark.parametrize("steps", [1, 2, 3, 4, 6, 7, 8, 9])
def test_other_numbers_of_iterations(q, steps):
    rng = np.random.default_rng(steps)
    for out in (F32, BF16):
        for rows, cols in ((70, 200), (200, 70)):
            x = torch.from_numpy(gradient(rng, rows, cols)).cuda()
            want, most = allowance(host(x), steps, out)
            assert np.linalg.norm(host(q.qopt_orthogonalize(x, steps=steps, out_dtype=out)) - want) <= most


def reference(x):
    """The definition in binary64 on the GPU."""
    a, b, c = muon.COEFFICIENTS
    x = x.double() / torch.linalg.vector_norm(x.double())
    tall = x.shape[0] > x.shape[1]
    x = x.t().contiguous() if tall else x
    for _ in range(5):
        g = x @ x.t().contiguous()
        x = a * x + (b * g + c * (g @ g)) @ x
    return x.t() if tall else x


@pytest.mark.parametrize("batch,rows,cols", [(1, 2048, 2100), (2, 1500, 4200), (1, 4400, 1200), (3, 2048, 2048), (1, 4096, 9000),
                                             (6, 4096, 300), (1, 5000, 5000)])
def test_large_matrices(q, batch, rows, cols):
    """Tiles of both sizes, several matrices of one launch.  Normal entries: 3e-7 is what rounding to 22 bits
    moves such matrices by, 1.2e-3 the single 11 bits of a bf16 destination's last iterations (the model
    at 512 x 1376), eight times that as elsewhere, and the sums."""
    say(f"orthogonalize {batch}x{rows}x{cols}")
    g = torch.Generator(device="cuda").manual_seed(rows)
    x = torch.randn(batch, rows, cols, generator=g, device="cuda") * 1e-3
    for out, size in ((F32, 3e-7), (BF16, 1.2e-3)):
        got = q.qopt_orthogonalize(x, out_dtype=out)
        for i in range(batch):
            want = reference(x[i])
            off = ((got[i].double() - want).norm() / want.norm()).item()
            assert off <= 8 * size * (1 + max(rows, cols) ** 0.5 / 8 * (out == F32)) + HALF[out], (out, i, off)


@pytest.mark.parametrize("rows,cols", [(64, 20000), (1, 100000), (100000, 1), (40, 131072), (300, 30000), (129, 2000)])
def test_long_sums(q, rows, cols):
    """Few tiles whose sums are long: shared between many workgroups."""
    say(f"orthogonalize {rows}x{cols}")
    g = torch.Generator(device="cuda").manual_seed(cols)
    x = torch.randn(rows, cols, generator=g, device="cuda") * 1e-3
    want = reference(x)
    for out, size in ((F32, 3e-7), (BF16, 1.2e-3)):
        got = q.qopt_orthogonalize(x, out_dtype=out)
        off = ((got.double() - want).norm() / want.norm()).item()
        assert off <= 8 * size * (1 + max(rows, cols) ** 0.5 / 8 * (out == F32)) + HALF[out], (out, off)
        assert torch.equal(got, q.qopt_orthogonalize(x, out_dtype=out))


def test_matrices_of_many_sizes_in_one_step(q):
    """Tiles whose sums are of different lengths in one launch."""
    g = torch.Generator(device="cuda").manual_seed(1)
    for shapes in ([(2048, 2048), (2048, 8192), (300, 9000), (100, 64)], [(1500, 1400), (257, 6000), (4000, 700), (130, 129), (9, 7000)]):
        ts = [tuple(torch.randn(s, generator=g, device="cuda") * v for v in (0.02, 1e-3, 1e-3)) for s in shapes]
        copies = [tuple(x.clone() for x in t) for t in ts]
        q.qopt_muon32bit_step(ts, lr=1.0, momentum=0.5, weight_decay=0.0, nesterov=False)
        for t, c in zip(ts, copies):
            assert torch.equal(t[2], c[2] * 0.5 + c[1] * 0.5)
            o = reference(t[2])
            r = float(muon.rate(1.0, *t[0].shape, "original"))
            off = ((t[0].double() - (c[0].double() - o * r)).norm() / (o.norm() * r)).item()
            # the parameter's own rounding is at most as large as it is next to the update
            own = 4 * 2.0 ** -24 * (1 + (c[0].norm() / (o.norm() * r)).item())
            assert off <= 8 * 3e-7 * (1 + max(t[0].shape) ** 0.5 / 8) + own, (t[0].shape, off)


def test_a_batch_is_its_matrices(q):
    """More matrices than one lot takes, and each as it is by itself."""
    rng = np.random.default_rng(4)
    for rows, cols, n in ((40, 60, 37), (130, 70, 5)):
        x = torch.from_numpy(np.stack([gradient(rng, rows, cols) for _ in range(n)])).cuda()
        got = q.qopt_orthogonalize(x)
        for i in range(n):
            assert torch.equal(got[i], q.qopt_orthogonalize(x[i]))
        assert torch.equal(q.qopt_orthogonalize(x.view(1, n, rows, cols))[0], got)


def test_out_and_what_lies_around_it(q):
    rng = np.random.default_rng(5)
    for dtype in (F32, BF16):
        for rows, cols in ((99, 301), (301, 99), (7, 3)):
            x = torch.from_numpy(gradient(rng, rows, cols)).cuda()
            want = q.qopt_orthogonalize(x, out_dtype=dtype)
            for off in (0, 1, 3):  # unaligned destinations, and their neighbours
                buf = torch.full((rows * cols + 8,), 7.0, dtype=dtype, device="cuda")
                out = buf[off:off + rows * cols].view(rows, cols)
                assert q.qopt_orthogonalize(x, out_dtype=dtype, out=out) is out
                assert torch.equal(out, want) and bool((buf[:off] == 7).all()) and bool((buf[off + rows * cols:] == 7).all())
                src = torch.zeros(rows * cols + 8, device="cuda")[off:off + rows * cols].view(rows, cols)
                src.copy_(x)
                assert torch.equal(q.qopt_orthogonalize(src, out_dtype=dtype), want)
    with pytest.raises(ValueError):
        q.qopt_orthogonalize(x, out=x)
    with pytest.raises(ValueError):
        q.qopt_orthogonalize(x, out=torch.empty(3, 7, device="cuda").t())


def test_zeros_sizes_and_what_is_not_finite(q):
    rng = np.random.default_rng(6)
    x = torch.from_numpy(np.stack([gradient(rng, 70, 90) for _ in range(6)])).cuda()
    want = q.qopt_orthogonalize(x)
    bad = x.clone()
    bad[1] = 0
    bad[2, 3, 4] = float("nan")
    bad[4, 69, 89] = float("inf")
    for dtype in (F32, BF16):
        got = q.qopt_orthogonalize(bad, out_dtype=dtype)
        assert not got[1].any() and got[2].isnan().all() and got[4].isnan().all()
        keep = [0, 3, 5]
        assert torch.equal(got[keep], q.qopt_orthogonalize(x, out_dtype=dtype)[keep])
    # squares that binary32 cannot hold, large and small (eps aside)
    for size in (1e30, 1e-30):
        got = q.qopt_orthogonalize(x * size, eps=1e-38)
        assert ((got - want).norm() / want.norm()).item() < 1e-5
    # under eps a matrix is divided by eps
    tiny = x[0] * 1e-8
    exact, most = allowance(host(tiny), 5, F32)
    assert np.linalg.norm(host(tiny)) < 1e-7
    assert np.linalg.norm(host(q.qopt_orthogonalize(tiny)) - exact) <= most
    for shape in ((0, 4, 5), (3, 0, 5), (3, 4, 0)):
        assert q.qopt_orthogonalize(torch.empty(shape, device="cuda")).shape == shape


# ------------------------------------------------------------------ steps

HP = dict(lr=2e-3, momentum=0.9, weight_decay=0.1)


def state_of(rng, rows, cols, bits, pdt, gdt):
    p = torch.from_numpy((rng.normal(size=(rows, cols)) * 0.02).astype(np.float32)).to("cuda", pdt)
    g = torch.from_numpy(gradient(rng, rows, cols)).to("cuda", gdt)
    m = gradient(rng, rows, cols)
    if bits == 32:
        return p, g, torch.from_numpy(m).cuda()
    codes, am = oracle.quantize_blockwise(m.ravel(), oracle.SIGNED)
    return p, g, torch.from_numpy(codes).cuda().view(rows, cols), torch.from_numpy(am).cuda()


def old_momentum(t):
    if len(t) == 3:
        return t[2].cpu().numpy()
    return oracle.dequantize_blockwise(t[2].cpu().numpy().ravel(), t[3].cpu().numpy(), oracle.SIGNED).reshape(t[0].shape)


def expected(t, hp, scale=None, nesterov=True, adjust="original"):
    """(new momentum, new parameter in binary64, how far it may be off)."""
    p, g = host(t[0]), t[1].float().cpu().numpy()
    with np.errstate(all="ignore"):
        m, u = muon.momentum(g, old_momentum(t), hp["momentum"], nesterov, scale)
    o, most = allowance(u, 5, t[0].dtype)
    r, d = float(muon.rate(hp["lr"], *p.shape, adjust)), float(muon.decay(hp["lr"], hp["weight_decay"]))
    want = p * d - o * r
    # four roundings of the two products and their difference, and the parameter's own
    size = np.linalg.norm(abs(p) + abs(o * r))
    return m, want, r * most + 4 * 2.0 ** -24 * size + HALF[t[0].dtype] * np.linalg.norm(want)


def check_step(t, m, want, most):
    off = np.linalg.norm(host(t[0]) - want)
    assert off <= most, (off, most)
    if len(t) == 3:
        assert np.array_equal(t[2].cpu().numpy(), m)
    else:
        codes, am = oracle.quantize_blockwise(m.ravel(), oracle.SIGNED)
        assert np.array_equal(t[3].cpu().numpy(), am)
        assert np.array_equal(t[2].cpu().numpy().ravel(), codes)


def run_step(q, bits, tensors, **kw):
    (q.qopt_muon8bit_step if bits == 8 else q.qopt_muon32bit_step)(tensors, **kw)


@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("pdt,gdt", [(F32, F32), (F32, BF16), (BF16, BF16), (BF16, F32)])
def test_step(q, bits, pdt, gdt):
    """Matrices of many shapes at once, blocks that end inside of one."""
    rng = np.random.default_rng(bits)
    shapes = [(33, 65), (64, 32), (1, 1), (300, 129), (129, 300), (2, 3000), (70, 70), (33, 700), (64, 64)]
    for kw in (dict(), dict(nesterov=False, adjust="match_rms_adamw"), dict(scale=0.37)):
        scale = kw.pop("scale", None)
        ts = [state_of(rng, r, c, bits, pdt, gdt) for r, c in shapes]
        want = [expected(t, HP, scale, **kw) for t in ts]
        gs = None if scale is None else torch.full((1,), scale, device="cuda")
        run_step(q, bits, ts, **HP, **kw, grad_scale=gs)
        for t, w in zip(ts, want):
            check_step(t, *w)


@pytest.mark.parametrize("bits", [8, 32])
def test_a_plan_stepped_again_and_again(q, bits):
    rng = np.random.default_rng(7)
    ts = [state_of(rng, r, c, bits, F32, F32) for r, c in ((50, 130), (64, 64))]
    plan = (q.qopt_muon8bit_plan if bits == 8 else q.qopt_muon32bit_plan)(ts)
    for _ in range(4):
        want = [expected(t, HP) for t in ts]
        run_step(q, bits, plan, **HP)
        for t, w in zip(ts, want):
            check_step(t, *w)
            t[1].copy_(torch.from_numpy(gradient(rng, *t[1].shape)))
    with pytest.raises(ValueError):
        run_step(q, 40 - bits, plan, **HP)


def test_what_lies_around_the_tensors_stays(q):
    """Unaligned matrices in larger buffers."""
    rng = np.random.default_rng(8)
    for bits in (8, 32):
        rows, cols = 37, 61
        n = rows * cols
        fresh = state_of(rng, rows, cols, bits, BF16, BF16)
        bufs, views = [], []
        for x in fresh:
            b = torch.full((x.numel() + 9,), 7, dtype=x.dtype, device="cuda")
            v = b[3:3 + x.numel()].view(x.shape)
            v.copy_(x)
            bufs.append(b), views.append(v)
        want = expected(tuple(views), HP)
        run_step(q, bits, [tuple(views)], **HP)
        check_step(tuple(views), *want)
        run_step(q, bits, [fresh], **HP)
        assert all(torch.equal(a, b) for a, b in zip(views, fresh))
        for b in bufs:
            assert bool((b[:3] == 7).all()) and bool((b[-6:] == 7).all())
        assert n == rows * cols


def test_gradients_that_are_not_finite_stay_in_their_matrix(q):
    rng = np.random.default_rng(9)
    for bits in (8, 32):
        ts = [state_of(rng, 40, 60, bits, F32, F32) for _ in range(3)]
        ts[1][1][5, 6] = float("nan")
        want = [expected(ts[i], HP) for i in (0, 2)]
        run_step(q, bits, ts, **HP)
        assert ts[1][0].isnan().all()
        check_step(ts[0], *want[0]), check_step(ts[2], *want[1])
        if bits == 8:  # as for the Adam step: a block with a NaN is stored as zeros
            assert ts[1][3][0].item() == 0 and not ts[1][2].view(-1)[:2048].any()


def test_zero_gradients_and_momentum(q):
    for bits in (8, 32):
        z = torch.zeros(50, 70, device="cuda")
        t = (torch.ones(50, 70, device="cuda"), z.clone(), z.clone()) if bits == 32 else \
            (torch.ones(50, 70, device="cuda"), z.clone(), z.to(torch.uint8), torch.zeros(2, device="cuda"))
        run_step(q, bits, [t], **HP)
        assert torch.equal(t[0], torch.full_like(t[0], float(muon.decay(2e-3, 0.1)))) and not t[2].any()


def test_refusals(q):
    rng = np.random.default_rng(10)
    a, b = state_of(rng, 20, 30, 32, F32, F32), state_of(rng, 20, 30, 32, F32, F32)
    for bad in ([a, a], [a, (a[0], b[1], b[2])], [a, (b[0], b[1], a[2])], [(a[0], a[0], a[2])]):
        with pytest.raises(ValueError):
            q.qopt_muon32bit_step(bad, **HP)
    with pytest.raises(TypeError):
        q.qopt_muon32bit_step([a, (b[0].bfloat16(), b[1], b[2])], **HP)
    with pytest.raises(ValueError):
        q.qopt_muon32bit_step([a], **HP, grad_scale=torch.ones(1))
    run_step(q, 32, [(a[0], a[1], a[2]), (b[0], a[1].clone(), b[2])], **HP)
    run_step(q, 32, [(torch.empty(0, 5, device="cuda"),) * 3, (torch.empty(3, 0, device="cuda"),) * 3], **HP)


def test_two_matrices_may_share_a_gradient(q):
    rng = np.random.default_rng(11)
    a, b = state_of(rng, 20, 30, 32, F32, F32), state_of(rng, 20, 30, 32, F32, F32)
    b = (b[0], a[1], b[2])
    want = [expected(t, HP) for t in (a, b)]
    q.qopt_muon32bit_step([a, b], **HP)
    check_step(a, *want[0]), check_step(b, *want[1])


def test_the_callers_stream_and_a_captured_step(q):
    rng = np.random.default_rng(12)
    for bits in (8, 32):
        ts = [state_of(rng, r, c, bits, BF16, BF16) for r, c in ((130, 200), (64, 300), (200, 130))]
        copies = [tuple(x.clone() for x in t) for t in ts]
        scale = torch.ones(1, device="cuda")
        plan = (q.qopt_muon8bit_plan if bits == 8 else q.qopt_muon32bit_plan)(ts)
        x = torch.from_numpy(gradient(rng, 90, 70)).cuda()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.stream(side):
            q.qopt_orthogonalize(x)
        torch.cuda.current_stream().wait_stream(side)
        with torch.cuda.graph(graph):
            run_step(q, bits, plan, **HP, grad_scale=scale)
            y = q.qopt_orthogonalize(x)
        for i in range(4):
            scale.fill_(0.5 + i)
            x.copy_(torch.from_numpy(gradient(rng, 90, 70)))
            for t, c in zip(ts, copies):
                t[1].copy_(torch.from_numpy(gradient(rng, *t[1].shape)))
                c[1].copy_(t[1])
            graph.replay()
            torch.cuda.synchronize()
            run_step(q, bits, copies, **HP, grad_scale=scale)
            for t, c in zip(ts, copies):
                assert all(torch.equal(s, w) for s, w in zip(t, c))
            assert torch.equal(y, q.qopt_orthogonalize(x))


def test_two_threads_at_once(q):
    rng = np.random.default_rng(13)
    jobs = [torch.from_numpy(gradient(rng, r, c)).cuda() for r, c in ((300, 400), (128, 900))]
    want = [q.qopt_orthogonalize(x) for x in jobs]
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(10):
                y = q.qopt_orthogonalize(jobs[i])
                torch.cuda.current_stream().synchronize()
                if not torch.equal(y, want[i]):
                    wrong.append(i)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert not wrong


# ------------------------------------------------------------------ the optimizer

def model(rng, dtype=F32, shapes=((96, 64), (40, 96), (64, 64), (8, 16))):
    return [torch.nn.Parameter(torch.from_numpy((rng.normal(size=s) * 0.02).astype(np.float32)).to("cuda", dtype)) for s in shapes]


def set_grads(rng, ps):
    for p in ps:
        p.grad = torch.from_numpy(gradient(rng, *p.shape)).to("cuda", p.dtype)


def test_optimizer(q):
    rng = np.random.default_rng(14)
    ps = model(rng)
    opt = q.Muon(ps, lr=2e-3, momentum=0.9, weight_decay=0.1, min_8bit_size=4096)
    for _ in range(3):
        set_grads(rng, ps)
        want = []
        for p in ps:
            st = opt.state[p]
            if not st:
                st = dict(m_codes=torch.zeros(p.numel(), dtype=torch.uint8, device="cuda"),
                          m_absmax=torch.zeros(-(-p.numel() // 2048), device="cuda")) if p.numel() >= 4096 \
                    else dict(momentum_buffer=torch.zeros_like(p))
                opt.state.pop(p)
            want.append(expected((p, p.grad, *st.values()), HP))
        opt.step()
        for p, w in zip(ps, want):
            st = opt.state[p]
            check_step((p, p.grad, *(st[k] for k in (("m_codes", "m_absmax") if "m_codes" in st else ("momentum_buffer",)))), *w)
    assert sorted("m_codes" in opt.state[p] for p in ps) == [False, False, True, True]  # 3840 and 128 elements; 4096 and 6144


def test_optimizer_groups_and_state_dict(q):
    rng = np.random.default_rng(15)
    ps = model(rng, BF16)
    make = lambda ps: q.Muon([dict(params=ps[:2]), dict(params=ps[2:], state_bits=32, lr=5e-3, adjust="match_rms_adamw")],  # noqa: E731
                             lr=1e-3, min_8bit_size=1)
    opt = make(ps)
    set_grads(rng, ps)
    opt.step()
    twin = [torch.nn.Parameter(p.detach().clone()) for p in ps]
    other = make(twin)
    other.load_state_dict(opt.state_dict())
    for _ in range(2):
        set_grads(rng, ps)
        for p, t in zip(ps, twin):
            t.grad = p.grad.clone()
        opt.step(), other.step(grad_scale=torch.ones(1, device="cuda"))
        assert all(torch.equal(p, t) for p, t in zip(ps, twin))
    for p, t in zip(ps, twin):
        a, b = opt.state[p], other.state[t]
        assert sorted(a) == sorted(b) and all(torch.equal(a[k], b[k]) and a[k].dtype == b[k].dtype for k in a)
    broken = opt.state_dict()
    broken["state"][0]["m_codes"] = broken["state"][0]["m_codes"][:5]
    with pytest.raises(ValueError):
        make(twin).load_state_dict(broken)


def test_torch_muon_state_converts(q):
    if not hasattr(torch.optim, "Muon"):
        pytest.skip("this torch has no Muon")
    rng = np.random.default_rng(16)
    ps = model(rng)
    ref = torch.optim.Muon(ps, lr=3e-3, momentum=0.8, weight_decay=0.05, nesterov=False, adjust_lr_fn="match_rms_adamw")
    set_grads(rng, ps)
    ref.step()
    twin = [torch.nn.Parameter(p.detach().clone()) for p in ps]
    opt = q.Muon(twin, state_bits=32)
    opt.load_fp32_muon_state(ref.state_dict())
    g = opt.param_groups[0]
    assert (g["lr"], g["momentum"], g["weight_decay"], g["nesterov"], g["adjust"]) == (3e-3, 0.8, 0.05, False, "match_rms_adamw")
    for p, t in zip(ps, twin):
        assert torch.equal(ref.state[p]["momentum_buffer"], opt.state[t]["momentum_buffer"])
    back = torch.optim.Muon(twin)
    back.load_state_dict(opt.fp32_muon_state_dict())
    for p, t in zip(ps, twin):
        assert torch.equal(ref.state[p]["momentum_buffer"], back.state[t]["momentum_buffer"])
    coded = q.Muon(twin, min_8bit_size=1)
    coded.load_fp32_muon_state(ref.state_dict())
    for p, t in zip(ps, twin):
        codes, am = oracle.quantize_blockwise(ref.state[p]["momentum_buffer"].cpu().numpy().ravel(), oracle.SIGNED)
        assert np.array_equal(coded.state[t]["m_codes"].cpu().numpy(), codes)
    with pytest.raises(ValueError):
        opt.load_fp32_muon_state(torch.optim.Muon(twin, ns_coefficients=(2.0, -1.5, 0.5)).state_dict())


def test_optimizer_refuses_before_any_state(q):
    rng = np.random.default_rng(17)
    ps = model(rng)
    opt = q.Muon([dict(params=ps[:2]), dict(params=ps[2:])], min_8bit_size=1)
    set_grads(rng, ps)
    before = [p.detach().clone() for p in ps]
    opt.param_groups[1]["lr"] = -1.0
    with pytest.raises(q.QoptError):
        opt.step()
    opt.param_groups[1]["lr"] = 1e-3
    ps[3].grad = ps[3].grad.t().contiguous().t()
    with pytest.raises(RuntimeError):
        opt.step()
    ps[3].grad = ps[3].grad.contiguous()
    ps[3].data = ps[2].data.view(-1)[:128].view(8, 16)  # two of one list
    with pytest.raises(ValueError):
        opt.step()
    assert not opt.state and all(torch.equal(p, b) for p, b in zip(ps[:2], before))


def test_a_captured_step_begins_no_state(q, monkeypatch):
    rng = np.random.default_rng(19)
    ps = model(rng)
    opt = q.Muon(ps, min_8bit_size=1)
    set_grads(rng, ps)
    before = [p.detach().clone() for p in ps]
    with monkeypatch.context() as m:
        m.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
        with pytest.raises(RuntimeError, match="capture"):
            opt.step()
        assert not any(opt.state.values()) and all(torch.equal(p, b) for p, b in zip(ps, before))
    opt.step()
    assert all(opt.state[p] for p in ps)


def test_an_optimizers_step_replayed(q):
    """Three replays of a captured step, each with its own gradients and eager work between them, against eager steps."""
    rng = np.random.default_rng(20)
    ps, twin = model(rng), None
    opt = q.Muon(ps, lr=2e-3, min_8bit_size=4096)
    set_grads(rng, ps)
    opt.step()
    twin = [torch.nn.Parameter(p.detach().clone()) for p in ps]
    other = q.Muon(twin, lr=2e-3, min_8bit_size=4096)
    other.load_state_dict(opt.state_dict())
    grads = [p.grad for p in ps]
    kept = [p.detach().clone() for p in ps]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        opt.step()
    assert all(torch.equal(p, k) for p, k in zip(ps, kept))  # a capture steps nothing
    for _ in range(3):
        for p, t, g in zip(ps, twin, grads):
            g.copy_(torch.from_numpy(rng.standard_normal(p.shape)))
            t.grad = g.clone()
        other.step()
        graph.replay()
        torch.cuda.synchronize()
        for p, t in zip(ps, twin):
            a, b = opt.state[p], other.state[t]
            assert torch.equal(p, t) and all(torch.equal(a[k], b[k]) for k in a)


def test_a_block_trains_with_all_of_them(q):
    """A feed-forward block's step: normalised, through two 4-bit products, matrices by Muon, the norm's vectors
    by AdamW.  The same step from the parts called by hand gives the same parameters."""
    torch.manual_seed(0)

    class Block(torch.nn.Module):
        def __init__(self):
            super().__init__()
            self.norm = q.LayerNorm(128)
            self.up, self.down = q.Fp4Linear(128, 320, seed=1), q.Fp4Linear(320, 128, seed=2)

        def forward(self, x):
            return x + self.down(torch.nn.functional.gelu(self.up(self.norm(x))))

    blocks = [Block(), Block()]
    blocks[1].load_state_dict(blocks[0].state_dict())
    x, dy = torch.randn(70, 128, device="cuda"), torch.randn(70, 128, device="cuda")
    b = blocks[0]
    muons, adam = q.Muon([b.up.weight, b.down.weight], lr=0.01), q.AdamW(b.norm.parameters(), lr=0.01, state_bits=32)
    y = b(x)
    y.backward(dy)
    muons.step(), adam.step()
    c = blocks[1]
    n, nw, nb = x, c.norm.weight, c.norm.bias
    h0, mean, rstd = q.qopt_layer_norm_forward(n, nw.detach(), nb.detach())
    h1 = q.qopt_fp4_linear(h0, *c.up.pack()).requires_grad_()
    h2 = torch.nn.functional.gelu(h1)
    assert torch.equal(y, x + q.qopt_fp4_linear(h2.detach(), *c.down.pack()))

    def gradients(x, w, dy):
        dx = q.qopt_fp8_matmul(*q.qopt_fp8_quantize(dy), *q.qopt_fp8_quantize(w, tiles=True, normal=False, transposed=True), F32)
        t = dict(normal=False, transposed=True)
        return dx, q.qopt_fp8_matmul(*q.qopt_fp8_quantize(dy, **t), *q.qopt_fp8_quantize(x, **t), F32)

    d2, down = gradients(h2.detach(), c.down.weight.detach(), dy)
    d1 = torch.autograd.grad(h2, h1, d2)[0]
    d0, up = gradients(h0, c.up.weight.detach(), d1)
    _, gw, gb = q.qopt_layer_norm_backward(n, nw.detach(), mean, rstd, d0)
    with torch.no_grad():
        state = lambda p: (torch.zeros(p.numel(), dtype=torch.uint8, device="cuda"), torch.zeros(-(-p.numel() // 2048), device="cuda"))  # noqa: E731
        ps = (c.up.weight.detach(), c.down.weight.detach())
        q.qopt_muon8bit_step([(p, g, *state(p)) for p, g in zip(ps, (up, down))], lr=0.01, momentum=0.95, weight_decay=0.1)
        q.qopt_adamw32bit_step([(p.detach(), g, torch.zeros_like(p), torch.zeros_like(p)) for p, g in ((nw, gw), (nb, gb))],
                               lr=0.01, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=1e-2, step=1)
    for s, t in zip(b.parameters(), c.parameters()):
        assert torch.equal(s, t)
