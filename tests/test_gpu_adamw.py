"""GPU parity of the AdamW steps (8-bit and 32-bit moments) against the oracle: codes, block
maxima, fp32 moments and fp32 / bf16 parameters bit for bit, since both sides round the
same binary32 operations in the same order."""

import copy
import threading

import numpy as np
import pytest
import torch

import oracle
from workloads import BLOCK

pytestmark = pytest.mark.gpu
HP = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.1)
PAIRS = [("f32", "f32"), ("f32", "bf16"), ("bf16", "f32"), ("bf16", "bf16")]
SIZES = [1, 7, 0, 2047, 2048, 2049, 50257, 3 * 2048 + 5, 17 * 2048]


def say(msg):
    print(msg, flush=True)


@pytest.fixture(scope="module")
def q():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import block_wise_bit_adam8bit_amd as q
    torch.cuda.set_device(0)
    return q


def to_dev(a, dtype="f32"):
    if dtype == "bf16":
        return torch.from_numpy(a.view(np.int16).copy()).cuda().view(torch.bfloat16)
    return torch.from_numpy(np.array(a)).cuda()


def to_host(t):
    if t.dtype == torch.bfloat16:
        return t.detach().reshape(-1).view(torch.int16).cpu().numpy().view(np.uint16)
    return t.detach().reshape(-1).cpu().numpy()


def bits(a):
    return a.view(np.uint32) if a.dtype == np.float32 else a


def same(got, want, what):
    bad = np.nonzero(bits(got) != bits(want))[0]
    assert bad.size == 0, f"{what}: {bad.size} differ, first at {bad[:4]}"


def draws(n, dtype, rng, std):
    x = rng.normal(0, std, n).astype(np.float32)
    if n and std < 0.01:
        x[rng.choice(n, size=max(1, n // 500), replace=False)] *= 100
    return oracle.f32_to_bf16_rne(x) if dtype == "bf16" else x


def zero_state(n, nbits):
    if nbits == 32:
        return [np.zeros(n, np.float32), np.zeros(n, np.float32)]
    nb = -(-n // BLOCK)
    return [np.zeros(n, np.uint8), np.zeros(n, np.uint8), np.zeros(nb, np.float32),
            np.zeros(nb, np.float32)]


def oracle_step(nbits):
    return oracle.adamw32bit_step if nbits == 32 else oracle.adamw8bit_step


def own_step(q, nbits):
    return q.qopt_adamw32bit_step if nbits == 32 else q.qopt_adamw8bit_step


def run_parity(q, nbits, sizes, pdt, gdt, steps, seed, hp=HP, scale=None, place=None, grads=None):
    """Every element of every tensor against the oracle, after every step."""
    rng = np.random.default_rng(seed)
    hp_p = [draws(n, pdt, rng, 0.02) for n in sizes]
    hs = [zero_state(n, nbits) for n in sizes]
    place = place or (lambda a, dtype: to_dev(a, dtype))
    dp = [place(p, pdt) for p in hp_p]
    ds = [[place(x, "f32") for x in s] for s in hs]
    gs = None if scale is None else torch.full((1,), scale, device="cuda")
    for step in range(1, steps + 1):
        hg = [(grads or draws)(n, gdt, rng, 1e-3) for n in sizes]
        dg = [place(g, gdt) for g in hg]
        own_step(q, nbits)([(dp[i], dg[i], *ds[i]) for i in range(len(sizes))], step=step,
                           grad_scale=gs, **hp)
        torch.cuda.synchronize()
        for i, n in enumerate(sizes):
            with np.errstate(all="ignore"):
                out = oracle_step(nbits)(hp_p[i], hg[i], *hs[i], step=step, grad_scale=scale,
                                         param_dtype=pdt, grad_dtype=gdt, **hp)
            hp_p[i], hs[i] = out[0], list(out[1:])
            what = f"{nbits}-bit {pdt}/{gdt} tensor {i} n={n} step {step}"
            same(to_host(dp[i]), hp_p[i], "param " + what)
            for k, (a, b) in enumerate(zip(ds[i], hs[i])):
                same(to_host(a), b, f"state {k} " + what)


@pytest.mark.parametrize("scale", [None, 0.37])
@pytest.mark.parametrize("pdt,gdt", PAIRS)
@pytest.mark.parametrize("nbits", [8, 32])
def test_dtypes_and_tails(q, nbits, pdt, gdt, scale):
    say(f"{nbits} {pdt}/{gdt} scale {scale}")
    run_parity(q, nbits, SIZES, pdt, gdt, 3, 7, scale=scale)


@pytest.mark.parametrize("nbits", [8, 32])
def test_many_small_tensors(q, nbits):
    sizes = [int(s) for s in np.random.default_rng(3).integers(0, 5000, 150)]
    say(f"{len(sizes)} tensors")
    run_parity(q, nbits, sizes, "f32", "bf16", 2, 4)


@pytest.mark.parametrize("pdt,gdt", PAIRS)
@pytest.mark.parametrize("nbits", [8, 32])
def test_views_at_odd_offsets(q, nbits, pdt, gdt):
    """Parameters, gradients and state one element into their buffers, on which wide
    accesses would be misaligned, with guard values on both sides left as they were."""
    guards = []

    def place(a, dtype):
        t = to_dev(a, dtype)
        buf = torch.full((t.numel() + 2,), 77, dtype=t.dtype, device="cuda")
        buf[1:-1] = t
        guards.append(buf)
        return buf[1:-1]

    run_parity(q, nbits, [2048, 6149, 3], pdt, gdt, 2, 5, place=place)
    for b in guards:
        assert float(b[0]) == 77 and float(b[-1]) == 77


@pytest.mark.parametrize("nbits", [8, 32])
@pytest.mark.parametrize("pdt", ["f32", "bf16"])
@pytest.mark.parametrize("hp", [dict(HP, beta1=0.0, beta2=0.0, weight_decay=0.0),
                                dict(HP, lr=5e-2, beta1=0.5, beta2=0.75, eps=1e-6, weight_decay=1.5),
                                dict(HP, eps=0.0, beta2=0.9999), dict(HP, eps=1e-20),
                                dict(HP, eps=1e-40), dict(HP, lr=4e6), dict(HP, lr=0.0)])
def test_hyperparameters(q, nbits, pdt, hp):
    """Step sizes and epsilons that switch the bf16 short path off, or make it fall back."""
    def grads(n, dtype, rng, std):
        g = draws(n, "f32", rng, std)
        if hp["eps"]:  # down to gradients whose squares underflow (0 / 0 without an epsilon)
            g[: n // 3] *= np.float32(10.0) ** rng.uniform(-25, 0, n // 3).astype(np.float32)
        return oracle.f32_to_bf16_rne(g) if dtype == "bf16" else g

    say(f"{nbits} {pdt} {hp}")
    run_parity(q, nbits, [2 ** 17 + 333], pdt, "bf16", 3, 12, hp=hp, grads=grads)


@pytest.mark.parametrize("pdt,gdt", PAIRS)
def test_without_decay_the_8bit_step_is_adam8bits(q, pdt, gdt):
    rng = np.random.default_rng(8)
    n = 9 * 2048 + 33
    p = to_dev(draws(n, pdt, rng, 0.02), pdt)
    one = torch.ones(1, device="cuda")
    a = [p.clone(), *(to_dev(x) for x in zero_state(n, 8))]
    b = [x.clone() for x in a]
    hp = {k: v for k, v in HP.items() if k != "weight_decay"}
    for step in range(1, 4):
        g = to_dev(draws(n, gdt, rng, 1e-3), gdt)
        q.qopt_adam8bit_step([(a[0], g, *a[1:])], step=step, **hp)
        q.qopt_adamw8bit_step([(b[0], g, *b[1:])], step=step, weight_decay=0.0, grad_scale=one, **hp)
        for x, y in zip(a, b):
            assert torch.equal(x, y)


@pytest.mark.parametrize("scale", [None, 0.37])
@pytest.mark.parametrize("eps", [1e-8, 0.0])
@pytest.mark.parametrize("pdt,gdt", PAIRS)
def test_large_and_small_8bit_steps_agree(q, pdt, gdt, eps, scale):
    """A step of many blocks leaves the bits that steps of its tensors one by one leave, which
    another kernel takes: odd lengths and offsets, zero, subnormal and non-finite blocks."""
    rng = np.random.default_rng(21)
    sizes = SIZES + [1400 * BLOCK] * 3 + [5 * BLOCK + 3]
    sets = []
    for i, n in enumerate(sizes):
        p, g = draws(n, pdt, rng, 0.02), draws(n, gdt, rng, 1e-3)
        m, v = rng.integers(0, 256, n).astype(np.uint8), rng.integers(0, 256, n).astype(np.uint8)
        am, av = (np.abs(rng.normal(0, s, -(-n // BLOCK))).astype(np.float32) for s in (1e-3, 1e-6))
        if n == 17 * BLOCK:
            gf = g if gdt == "f32" else oracle.bf16_to_f32(g)
            gf = gf.copy()
            gf[5], gf[3 * BLOCK], gf[4 * BLOCK + 9] = np.inf, np.nan, 1e30
            gf[6 * BLOCK:8 * BLOCK] = 0
            g = oracle.f32_to_bf16_rne(gf) if gdt == "bf16" else gf
            am[6], av[6], am[9], av[9] = 0, 0, 1e-40, 1e-42
        sets.append([to_dev(p, pdt), to_dev(g, gdt), to_dev(m), to_dev(v), to_dev(am), to_dev(av)])
    # the last tensor one element into its buffers
    for k in range(4):
        buf = torch.empty(sizes[-1] + 1, dtype=sets[-1][k].dtype, device="cuda")
        buf[1:] = sets[-1][k]
        sets[-1][k] = buf[1:]
    other = [[t.clone() for t in s] for s in sets]
    gs = None if scale is None else torch.full((1,), scale, device="cuda")
    hp = dict(HP, eps=eps)
    for step in (1, 2, 3):
        q.qopt_adamw8bit_step([tuple(s) for s in sets], step=step, grad_scale=gs, **hp)
        for s in other:
            q.qopt_adamw8bit_step([tuple(s)], step=step, grad_scale=gs, **hp)
        for n, x, y in zip(sizes, sets, other):
            for k, (a, b) in enumerate(zip(x, y)):
                if a.is_floating_point():  # a NaN's sign and payload included
                    a, b = (t.view(torch.int32 if t.dtype == torch.float32 else torch.int16) for t in (a, b))
                assert torch.equal(a, b), (step, n, k)


@pytest.mark.parametrize("nbits", [8, 32])
def test_non_finite_gradients(q, nbits):
    """NaN and infinities stay within their block (8-bit state: it is stored as zeros) or
    their element (32-bit state)."""
    def grads(n, dtype, rng, std):
        g = draws(n, "f32", rng, std)
        g[5], g[3000], g[5000] = np.nan, np.inf, -np.inf
        return oracle.f32_to_bf16_rne(g) if dtype == "bf16" else g

    rng = np.random.default_rng(1)
    n = 4 * 2048
    p, g = draws(n, "f32", rng, 0.02), grads(n, "f32", rng, 1e-3)
    st = zero_state(n, nbits)
    d = [to_dev(p), to_dev(g), *(to_dev(x) for x in st)]
    own_step(q, nbits)([tuple(d)], step=1, **HP)
    with np.errstate(all="ignore"):
        ref = oracle_step(nbits)(p, g, *st, step=1, **HP)
    for got, want in zip([d[0], *d[2:]], ref):
        got = to_host(got)
        if got.dtype == np.float32:
            assert np.array_equal(np.isnan(got), np.isnan(want))
            fine = ~np.isnan(want)
            same(got[fine], want[fine], "finite values")
        else:
            same(got, want, "codes")


@pytest.mark.parametrize("nbits", [8, 32])
def test_steps_a_captured_graph_replays(q, nbits):
    """A captured step, replayed with eager steps and synchronisations between the replays
    and the clipping factor changed on the device: every replay is the eager step.  The
    bf16 call has more than one launch, which outside a capture use a second stream."""
    rng = np.random.default_rng(2)
    sizes = [2048 * 60] * 50 + [2049] * 20
    p = [to_dev(draws(n, "bf16", rng, 0.02), "bf16") for n in sizes]
    st = [[to_dev(x) for x in zero_state(n, nbits)] for n in sizes]
    g = [to_dev(draws(n, "bf16", rng, 1e-3), "bf16") for n in sizes]
    gs = torch.ones(1, device="cuda")
    items = [(p[i], g[i], *st[i]) for i in range(len(sizes))]
    ref = [tuple(x.clone() for x in t) for t in items]
    step, make = own_step(q, nbits), {8: q.qopt_adamw8bit_plan, 32: q.qopt_adamw32bit_plan}[nbits]
    plan, eager = make(items), make(ref)
    for pl in (plan, eager):  # the warm-up that a capture wants, on both
        step(pl, step=3, grad_scale=gs, **HP)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(plan, step=3, grad_scale=gs, **HP)
    for r in range(4):
        gs.fill_(1.0 / (r + 1))
        graph.replay()
        step(eager, step=3, grad_scale=gs, **HP)
        torch.cuda.synchronize()
        for a, b in zip(items, ref):
            for x, y in zip(a, b):
                assert torch.equal(x, y), f"replay {r}"


@pytest.mark.parametrize("nbits", [8, 32])
def test_runs_on_the_callers_stream(q, nbits):
    """A step on a side stream, queued behind long products and the copies of its inputs."""
    rng = np.random.default_rng(6)
    n = 64 * 2048 + 9
    p, g = draws(n, "f32", rng, 0.02), draws(n, "f32", rng, 1e-3)
    d = [to_dev(x) for x in (np.zeros_like(p), np.zeros_like(g), *zero_state(n, nbits))]
    src = [to_dev(p), to_dev(g)]
    big = torch.randn(4096, 4096, device="cuda")
    gs = torch.zeros(1, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(6):
            big = big @ big * 1e-2
        d[0].copy_(src[0]), d[1].copy_(src[1]), gs.fill_(0.5)
        own_step(q, nbits)([tuple(d)], step=1, grad_scale=gs, **HP)
    torch.cuda.synchronize()
    ref = oracle_step(nbits)(p, g, *zero_state(n, nbits), step=1, grad_scale=0.5, **HP)
    for got, want in zip([d[0], *d[2:]], ref):
        same(to_host(got), want, "side stream")


def test_steps_from_two_threads(q):
    rng = np.random.default_rng(16)
    n = 300 * 2048 + 11
    jobs = []
    for nbits in (8, 32):
        p, g = draws(n, "bf16", rng, 0.02), draws(n, "bf16", rng, 1e-3)
        jobs.append((nbits, p, g, [to_dev(p, "bf16"), to_dev(g, "bf16"),
                                   *(to_dev(x) for x in zero_state(n, nbits))]))
    errors = []

    def work(nbits, d):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for step in range(1, 6):
                    own_step(q, nbits)([tuple(d)], step=step, **HP)
                torch.cuda.current_stream().synchronize()
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    torch.cuda.synchronize()
    ts = [threading.Thread(target=work, args=(j[0], j[3])) for j in jobs]
    [t.start() for t in ts], [t.join() for t in ts]
    assert not errors
    for nbits, p, g, d in jobs:
        ref = [p, *zero_state(n, nbits)]
        for step in range(1, 6):
            ref = list(oracle_step(nbits)(ref[0], g, *ref[1:], step=step, param_dtype="bf16",
                                          grad_dtype="bf16", **HP))
        for got, want in zip([d[0], *d[2:]], ref):
            same(to_host(got), want, f"{nbits}-bit thread")


def test_32bit_moments_past_32_bit_offsets(q):
    """One tensor of 2^32 + 2 * 2048 + 5 elements (and so past 2^31 and 2^32 elements and
    bytes), checked at both ends and around those offsets."""
    n = 2 ** 32 + 2 * 2048 + 5
    say(f"n={n}")
    p = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    g = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    m = torch.zeros(n, device="cuda")
    v = torch.zeros(n, device="cuda")
    spots = [0, 2 ** 29 - 1024, 2 ** 30 - 1024, 2 ** 31 - 1024, 2 ** 32 - 1024, n - 2048]
    rng = np.random.default_rng(4)
    host = []
    for o in spots:
        hp_, hg = draws(2048, "bf16", rng, 0.02), draws(2048, "bf16", rng, 1e-3)
        p[o:o + 2048], g[o:o + 2048] = to_dev(hp_, "bf16"), to_dev(hg, "bf16")
        host.append((hp_, hg))
    q.qopt_adamw32bit_step([(p, g, m, v)], step=1, **HP)
    for o, (hp_, hg) in zip(spots, host):
        ref = oracle.adamw32bit_step(hp_, hg, np.zeros(2048, np.float32), np.zeros(2048, np.float32),
                                     step=1, param_dtype="bf16", grad_dtype="bf16", **HP)
        for t, want in zip((p, m, v), ref):
            same(to_host(t[o:o + 2048]), want, f"at {o}")
    # nothing anywhere else moved: each nonzero moment lies in one of the spots
    inside = sum(int(torch.count_nonzero(m[o:o + 2048])) for o in spots)
    total = sum(int(torch.count_nonzero(c)) for c in m.split(2 ** 28))
    assert total == inside


def test_refused_lists(q):
    """Overlaps, wrong types, sizes and devices are refused before any launch."""
    n = 4096
    z = lambda dt=torch.float32, k=n, d="cuda": torch.zeros(k, dtype=dt, device=d)  # noqa: E731
    p, g, m, v = z(), z(), z(), z()
    codes = lambda: (z(torch.uint8), z(torch.uint8), z(k=2), z(k=2))  # noqa: E731
    plan32 = q.qopt_adamw32bit_plan([(p, g, m, v)])
    bad = [
        (ValueError, [(p, g, m, v), (p, z(), z(), z())]),        # a parameter listed twice
        (ValueError, [(p, g, m, m)]),                            # both moments in one buffer
        (ValueError, [(p, p, m, v)]),                            # the gradient is the parameter
        (ValueError, [(p[:2048], g[:2048], m[:2048], v[:2048]), (p[2047:], g[2047:], z(k=2049), z(k=2049))]),
        (TypeError, [(p, g, m.half(), v)]),
        (TypeError, [(p.half(), g, m, v)]),
        (TypeError, [(p, g, m, v), (z(torch.bfloat16), g, z(), z())]),
        (ValueError, [(p, g[:-1], m, v)]),
        (ValueError, [(p, g.view(64, 64).t(), m, v)]),
        (ValueError, [(p, z(d="cpu"), m, v)]),
    ]
    for err, items in bad:
        with pytest.raises(err):
            q.qopt_adamw32bit_step(items, step=1, **HP)
    with pytest.raises(ValueError):
        c = codes()
        q.qopt_adamw8bit_step([(p, g, c[0], c[0], c[2], c[3])], step=1, **HP)
    with pytest.raises(ValueError):
        q.qopt_adamw8bit_step(plan32, step=1, **HP)
    for gs in (z(k=2), z(torch.float64, 1), z(k=1, d="cpu")):
        with pytest.raises(ValueError):
            q.qopt_adamw32bit_step(plan32, step=1, grad_scale=gs, **HP)
    for change in (dict(weight_decay=-0.1), dict(weight_decay=float("nan")), dict(lr=float("inf")),
                   dict(beta1=1.0), dict(eps=-1.0)):
        with pytest.raises(q.QoptError):
            q.qopt_adamw32bit_step(plan32, step=1, **{**HP, **change})
    with pytest.raises(q.QoptError):
        q.qopt_adamw32bit_step(plan32, step=0, **HP)
    # one gradient may serve two parameters
    q.qopt_adamw32bit_step([(p, g, m, v), (z(), g, z(), z())], step=1, **HP)
    q.qopt_adamw32bit_step([], step=1, **HP)
    torch.cuda.synchronize()


# ------------------------------------------------------------------ the optimizer


def small_params(pdt=torch.float32):
    torch.manual_seed(0)
    shapes = [(64, 80), (80,), (4096,), (33, 7), (100, 41)]
    return [torch.nn.Parameter((torch.randn(s, device="cuda") * 0.02).to(pdt)) for s in shapes]


def set_grads(params, seed, dtype=None):
    g = torch.Generator(device="cuda").manual_seed(seed)
    for p in params:
        p.grad = (torch.randn(p.shape, device="cuda", generator=g) * 1e-3).to(p.dtype)


@pytest.mark.parametrize("pdt", [torch.float32, torch.bfloat16])
def test_optimizer_follows_the_oracle(q, pdt):
    """Mixed state kinds: by size within a group, by state_bits between groups."""
    params = small_params(pdt)
    name = "bf16" if pdt == torch.bfloat16 else "f32"
    opt = q.AdamW([dict(params=params[:4]), dict(params=params[4:], state_bits=32, weight_decay=0.0)],
                  lr=1e-3, weight_decay=0.1, min_8bit_size=4096)
    kinds = [8, 32, 8, 32, 32]
    ref = [[to_host(p.data).copy(), *zero_state(p.numel(), k)] for p, k in zip(params, kinds)]
    gs = torch.full((1,), 0.25, device="cuda")
    for step in range(1, 5):
        set_grads(params, step)
        opt.step(grad_scale=gs)
        for i, (p, k) in enumerate(zip(params, kinds)):
            hp = dict(HP, weight_decay=0.0 if i == 4 else 0.1)
            ref[i] = list(oracle_step(k)(ref[i][0], to_host(p.grad), *ref[i][1:], step=step,
                                         grad_scale=0.25, param_dtype=name, grad_dtype=name, **hp))
    for p, k, r in zip(params, kinds, ref):
        st = opt.state[p]
        assert st["step"] == 4 and ("m_codes" in st) == (k == 8)
        same(to_host(p.data), r[0], "param")
        keys = ("m_codes", "v_codes", "m_absmax", "v_absmax") if k == 8 else ("exp_avg", "exp_avg_sq")
        for key, want in zip(keys, r[1:]):
            same(to_host(st[key]), want, key)


def test_optimizer_resumes_and_converts(q, tmp_path):
    params = small_params()
    opt = q.AdamW(params, lr=1e-3, weight_decay=0.1, min_8bit_size=4096)
    for step in range(3):
        set_grads(params, step)
        opt.step()
    torch.save(opt.state_dict(), tmp_path / "opt.pt")
    twin = [torch.nn.Parameter(p.detach().clone()) for p in params]
    again = q.AdamW(twin, lr=5e-2, min_8bit_size=1 << 30)  # the saved kinds and settings win
    again.load_state_dict(torch.load(tmp_path / "opt.pt", weights_only=True))
    third = copy.deepcopy(opt)
    for step in range(3, 6):
        set_grads(params, step), set_grads(twin, step)
        opt.step(), again.step()
    for a, b in zip(params, twin):
        assert torch.equal(a, b)
    assert third.state
    # to torch.optim.AdamW and back: fp32 moments travel unchanged, coded ones as their values
    sd = opt.fp32_adam_state_dict()
    ref = torch.optim.AdamW([torch.nn.Parameter(p.detach().clone()) for p in params])
    ref.load_state_dict(sd)
    assert ref.param_groups[0]["weight_decay"] == 0.1 and ref.param_groups[0]["lr"] == 1e-3
    back = q.AdamW([torch.nn.Parameter(p.detach().clone()) for p in params], min_8bit_size=4096)
    back.load_fp32_adam_state(ref.state_dict())
    for a, b in zip(params, back.param_groups[0]["params"]):
        sa, sb = opt.state[a], back.state[b]
        assert sa["step"] == sb["step"] == 6 and set(sa) == set(sb)
        for k in set(sa) - {"step"}:
            assert torch.equal(sa[k], sb[k]), k
    assert back.param_groups[0]["weight_decay"] == 0.1
    # Adam8bit's state is taken over as it is
    a8 = q.Adam8bit([torch.nn.Parameter(torch.randn(5000, device="cuda"))])
    set_grads(a8.param_groups[0]["params"], 1)
    a8.step()
    w = q.AdamW([torch.nn.Parameter(a8.param_groups[0]["params"][0].detach().clone())])
    w.load_state_dict(a8.state_dict())
    set_grads(w.param_groups[0]["params"], 2)
    w.step()
    assert w.state[w.param_groups[0]["params"][0]]["step"] == 2


def test_optimizer_moves_with_its_tensors(q):
    """A gradient or parameter whose storage moves is found at its new place."""
    params = small_params()
    opt = q.AdamW(params, min_8bit_size=4096)
    ref = [torch.nn.Parameter(p.detach().clone()) for p in params]
    ropt = q.AdamW(ref, min_8bit_size=4096)
    for step in range(4):
        set_grads(params, step), set_grads(ref, step)
        if step == 2:
            for p in params:
                p.data = p.data.clone()
                p.grad = p.grad.clone()
        opt.step(), ropt.step()
    for a, b in zip(params, ref):
        assert torch.equal(a, b)


def test_optimizer_refuses(q):
    p = torch.nn.Parameter(torch.zeros(64, 64, device="cuda"))
    for bad in (dict(lr=-1.0), dict(eps=-1.0), dict(betas=(1.0, 0.9)), dict(weight_decay=-1.0),
                dict(state_bits=16)):
        with pytest.raises(ValueError):
            q.AdamW([p], **bad)
    opt = q.AdamW([p])
    p.grad = torch.zeros(64, 64, device="cuda").t()
    with pytest.raises(RuntimeError):
        opt.step()
    assert not opt.state or not opt.state[p]
    src = torch.optim.Adam([torch.nn.Parameter(torch.zeros(64, 64))], weight_decay=0.1)
    with pytest.raises(ValueError):
        opt.load_fp32_adam_state(src.state_dict())
    src = torch.optim.AdamW([torch.nn.Parameter(torch.zeros(64, 64))], amsgrad=True)
    with pytest.raises(ValueError):
        opt.load_fp32_adam_state(src.state_dict())


def test_optimizer_refuses_before_any_state(q):
    """Every group is looked over first: nothing has moved when one of them is refused."""
    good = torch.nn.Parameter(torch.ones(64, 64, device="cuda"))
    half = torch.nn.Parameter(torch.ones(64, 64, device="cuda", dtype=torch.float16))
    for p in (good, half):
        p.grad = torch.ones_like(p)
    opt = q.AdamW([dict(params=[good]), dict(params=[half])])
    with pytest.raises(TypeError):
        opt.step()
    assert not any(opt.state.values()) and bool((good == 1).all())
    opt = q.AdamW([good])
    with pytest.raises(ValueError):
        opt.step(grad_scale=torch.ones(1))
    assert not any(opt.state.values()) and bool((good == 1).all())


@pytest.mark.parametrize("nbits", [8, 32])
def test_a_plan_steps_the_memory_it_was_made_of(q, nbits):
    """A parameter given other memory leaves its plan with the old, which the plan keeps."""
    n = 5 * BLOCK + 3
    p = torch.nn.Parameter(torch.ones(n, device="cuda"))
    g = torch.ones(n, device="cuda")
    state = [to_dev(s) for s in zero_state(n, nbits)]
    plan = (q.qopt_adamw8bit_plan if nbits == 8 else q.qopt_adamw32bit_plan)([(p, g, *state)])
    old = p.data
    p.data = torch.full((n,), 3.0, device="cuda")
    own_step(q, nbits)(plan, step=1, **HP)
    assert bool((p == 3).all()) and bool((old < 1).all())
    del old
    other = [torch.full((n,), 5.0, device="cuda") for _ in range(20)]  # would take freed memory
    own_step(q, nbits)(plan, step=2, **HP)
    assert all(bool((o == 5).all()) for o in other) and bool((p == 3).all())


# ------------------------------------------------------------------ above the few blocks' and small steps' limits

# More blocks than the workgroup-per-block kernel takes (4096), and enough for a wave's whole runs.
MANY_BLOCKS = 20000


def equal_but_for_nans(a, b):
    if not a.is_floating_point():
        return torch.equal(a, b)
    nan = torch.isnan(a)
    bit = torch.int32 if a.dtype == torch.float32 else torch.int16
    return torch.equal(nan, torch.isnan(b)) and torch.equal(a.view(bit)[~nan], b.view(bit)[~nan])


@pytest.mark.parametrize("pdt,gdt", PAIRS)
@pytest.mark.parametrize("hp", [dict(HP, beta1=0.0, beta2=0.0, weight_decay=0.0),
                                dict(HP, lr=5e-2, beta1=0.5, beta2=0.75, eps=1e-6, weight_decay=1.5),
                                dict(HP, eps=0.0, beta2=0.9999), dict(HP, eps=1e-20),
                                dict(HP, eps=1e-40), dict(HP, lr=4e6), dict(HP, lr=0.0)])
def test_hyperparameters_of_many_blocks(q, pdt, gdt, hp):
    """The wave-per-block kernel with step sizes and epsilons that switch the bf16 short path off or make
    it look for subnormal second moments, scaled gradients and decay, from nonzero moments: sampled
    blocks against the oracle, every element against the other kernel, which steps of few blocks take."""
    say(f"{pdt}/{gdt} {hp}")
    n = MANY_BLOCKS * BLOCK + 333
    nb = MANY_BLOCKS + 1
    gen = torch.Generator(device="cuda").manual_seed(31)
    normal = lambda k, s: torch.randn(k, device="cuda", generator=gen) * s  # noqa: E731
    types = {"f32": torch.float32, "bf16": torch.bfloat16}
    p = normal(n, 0.02).to(types[pdt])
    codes = [torch.randint(0, 256, (n,), dtype=torch.uint8, device="cuda", generator=gen) for _ in range(2)]
    maxima = [normal(nb, s).abs() for s in (1e-3, 1e-6)]
    maxima[1][::7] = 0  # second moments that come from this step's gradients alone
    one = [p, None, *codes, *maxima]
    # the same by pieces of at most 2000 blocks, which the other kernel takes
    other = [None if t is None else t.clone() for t in one]
    sample = np.unique(np.concatenate([np.arange(9), np.random.default_rng(2).integers(0, MANY_BLOCKS, 60),
                                       MANY_BLOCKS - 1 - np.arange(4)]))
    at = torch.from_numpy((sample[:, None] * BLOCK + np.arange(BLOCK)).ravel()).cuda()
    blocks = torch.from_numpy(sample).cuda()
    tail = slice(MANY_BLOCKS * BLOCK, n)
    scale = torch.full((1,), 0.37, device="cuda")
    for step in (1, 2):
        g = normal(n, 1e-3)
        if hp["eps"]:  # down to gradients whose squares underflow (0 / 0 without an epsilon)
            g[: n // 3] *= 10.0 ** (torch.rand(n // 3, device="cuda", generator=gen) * -25)
        one[1] = g = g.to(types[gdt])
        parts = []
        for whole, b in ((True, blocks), (False, torch.tensor([MANY_BLOCKS], device="cuda"))):
            i = at if whole else torch.arange(tail.start, tail.stop, device="cuda")
            host = [to_host(t[i].contiguous()) for t in one[:4]] + [to_host(t[b]) for t in one[4:]]
            with np.errstate(all="ignore"):
                parts.append((i, b, oracle.adamw8bit_step(*host, step=step, grad_scale=0.37, param_dtype=pdt,
                                                          grad_dtype=gdt, **hp)))
        q.qopt_adamw8bit_step([tuple(one)], step=step, grad_scale=scale, **hp)
        for lo in range(0, nb, 2000):
            e, k = slice(lo * BLOCK, min(n, (lo + 2000) * BLOCK)), slice(lo, min(nb, lo + 2000))
            q.qopt_adamw8bit_step([(other[0][e], g[e], other[2][e], other[3][e], other[4][k], other[5][k])],
                                  step=step, grad_scale=scale, **hp)
        torch.cuda.synchronize()
        for i, b, want in parts:
            for k, (t, w) in enumerate(zip((one[0], *one[2:]), want)):
                got = t[b] if k > 2 else t[i]
                w = to_dev(w, "bf16") if w.dtype == np.uint16 else to_dev(w)
                assert equal_but_for_nans(got, w), f"oracle, step {step}, output {k}"
        for k in (0, 2, 3, 4, 5):
            assert equal_but_for_nans(one[k], other[k]), f"other kernel, step {step}, tensor {k}"


@pytest.mark.parametrize("scale", [None, 0.37])
@pytest.mark.parametrize("pdt,gdt", PAIRS)
def test_large_32bit_steps(q, pdt, gdt, scale):
    """Above 5 * 2^20 elements another instance of the kernel runs: tensors of odd lengths beside a large
    one, more of them than a launch holds, moments that are not zero."""
    say(f"{pdt}/{gdt} scale {scale}")
    sizes = [5 * 2 ** 20 + 5, 1025, 1, 0, 70003, *range(1000, 1100)]
    run_parity(q, 32, sizes, pdt, gdt, 3, 17, scale=scale)


@pytest.mark.parametrize("pdt,gdt", PAIRS)
def test_large_32bit_steps_at_odd_offsets(q, pdt, gdt):
    """... and one element into their buffers, where wide accesses would be misaligned."""
    guards = []

    def place(a, dtype):
        t = to_dev(a, dtype)
        buf = torch.full((t.numel() + 2,), 77, dtype=t.dtype, device="cuda")
        buf[1:-1] = t
        guards.append(buf)
        return buf[1:-1]

    run_parity(q, 32, [5 * 2 ** 20 + 1025, 1024, 3], pdt, gdt, 2, 18, scale=0.37, place=place)
    for b in guards:
        assert float(b[0]) == 77 and float(b[-1]) == 77
