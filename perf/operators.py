"""The operators of a training and serving step in 8 bits, as cases that can be timed and compared.

Two families:

* Matrix products of 8-bit floating point (e4m3) values with one power-of-two scale per block of 128:
  ``linear`` (activations times a packed weight, as a server calls it, from one token to a prompt) and
  ``train`` (the layer's forward and backward from a full-precision weight).
* AdamW steps over many tensors at once, with decoupled weight decay: ``adamw8`` (both moments held as
  block-wise dynamic-tree codes, blocks of 2048) and ``adamw32`` (both moments held in binary32).

``run`` computes the plain form with elementary torch operations, or, where ``own`` is true, makes the
calls of this repository's package.  ``exact`` computes the same results in binary64, written apart.

Definitions.  A block of 128 values x has the exponent e = the least integer with max|x| <= 448 * 2^e (over
the block's finite values, at least -127; e = 0 for a block of zeros) and stores e + 127 in one byte and
each x * 2^-e rounded to e4m3, nearest even.  Activations and upstream gradients have a block for every 128
consecutive values along the axis that is summed over, weights a block for every tile of 128 x 128.  A
product sums the values that the codes and scales stand for and is rounded once, to the output's type.

AdamW, for a gradient g scaled by s, step t, hyper-parameters in binary32:
    m = b1 m + (1 - b1) g s      v = b2 v + (1 - b2) (g s)^2
    p = p (1 - lr wd) - lr / (1 - b1^t) * m / (sqrt(v) / sqrt(1 - b2^t) + eps)
with one binary32 rounding per operation; in ``adamw8`` m and v are then requantized (nearest code of the
magnitude over the block's largest, distances in binary32, ties to the smaller code).
"""

import math
from fractions import Fraction

import numpy as np
import torch

own = False

BLOCK = 2048  # values per block of the 8-bit optimizer state
KBLOCK = 128  # values per block of the 8-bit products
DEVICE = "cuda"

HP = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.1, step=100)


# ------------------------------------------------------------------------------------------------ cases

_GPT_BLOCK = "2048,2048,4194304,4194304,4194304,4194304,2048,2048,16777216,16777216"
_LLAMA_BLOCK = "4096,16777216,16777216,16777216,16777216,4096,45088768,45088768,45088768"


def listed():
    return [
        # one token through an attention projection of the 7B set: latency and the weight's bytes
        dict(name="linear one token 4096x4096", op="linear", tokens=1, n=4096, k=4096, act="bf16"),
        # a small batch of sequences decoding through the 7B set's gate projection
        dict(name="linear 24 tokens 11008x4096", op="linear", tokens=24, n=11008, k=4096, act="bf16"),
        # the output head of the 1.3B set: an odd vocabulary, a few sequences
        dict(name="linear 7 tokens 50257x2048", op="linear", tokens=7, n=50257, k=2048, act="bf16"),
        # a prompt through the gate projection
        dict(name="linear 2048 tokens 11008x4096", op="linear", tokens=2048, n=11008, k=4096, act="bf16"),
        # a ragged batch through the 1.3B set's second feed-forward product; fp32 master weight, so its
        # gradient is fp32
        dict(name="train 1999 tokens 2048x8192", op="train", tokens=1999, n=2048, k=8192, act="bf16",
             weight="f32"),
        # the largest: 8192 tokens through the 7B set's gate projection, weight kept in bf16
        dict(name="train 8192 tokens 11008x4096", op="train", tokens=8192, n=11008, k=4096, act="bf16",
             weight="bf16"),
        # tiny and ragged tensors: latency, short blocks
        dict(name="adamw8 four odd tensors", op="adamw8", sizes="2049,50257,1,4097", param="f32", grad="f32",
             clip=False),
        # one transformer block of the 1.3B set, bf16 parameters in place, gradients clipped
        dict(name="adamw8 1.3B block bf16", op="adamw8", sizes=_GPT_BLOCK, param="bf16", grad="bf16",
             clip=True),
        # one transformer block of the 7B set, fp32 master weights and bf16 gradients
        dict(name="adamw8 7B block", op="adamw8", sizes=_LLAMA_BLOCK, param="f32", grad="bf16", clip=False),
        # every normalisation vector of the 1.3B set, which keep 32-bit moments: many small tensors
        dict(name="adamw32 98 norm vectors", op="adamw32", sizes=",".join(["2048"] * 98), param="f32",
             grad="bf16", clip=True),
        # odd lengths, bf16 parameters in place
        dict(name="adamw32 odd bf16", op="adamw32", sizes="1000003,77,65537,2048,3", param="bf16",
             grad="bf16", clip=False),
        # the 7B set's embedding table, which keeps 32-bit moments
        dict(name="adamw32 embedding", op="adamw32", sizes="131072000", param="f32", grad="bf16",
             clip=False),
    ]


def draw(rng):
    def spread(lo, hi):
        return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    op = rng.choice(["linear", "train", "adamw8", "adamw32"])
    if op in ("linear", "train"):
        n, k = spread(64, 11008), spread(64, 8192)
        most = 8192 * 11008 * 4096 // (n * k)
        case = dict(op=op, tokens=min(most, spread(1, 8192)), n=n, k=k, act=rng.choice(["bf16", "bf16", "f32"]))
        if op == "train":
            case["weight"] = rng.choice(["bf16", "f32"])
        return case
    sizes, left = [], 131072000
    for _ in range(spread(1, 60)):
        n = min(left, spread(1, 1 << 24))
        if n > 0:
            sizes.append(n)
            left -= n
    return dict(op=op, sizes=",".join(map(str, sizes)), param=rng.choice(["f32", "bf16"]),
                grad=rng.choice(["f32", "bf16"]), clip=rng.random() < 0.5)


_DTYPE = {"f32": torch.float32, "bf16": torch.bfloat16}
_BYTES = {"f32": 4, "bf16": 2}


def _blocks(sizes):
    return [-(-n // BLOCK) for n in sizes]


def work(case):
    if case["op"] in ("linear", "train"):
        m, n, k = case["tokens"], case["n"], case["k"]
        a = _BYTES[case["act"]]
        if case["op"] == "linear":
            kb = -(-k // KBLOCK)
            return {"bytes": m * k * a + n * k + kb * -(-n // KBLOCK) + m * n * a, "flops": 2 * m * n * k}
        # x, w and dy in; y, dx and dw out
        return {"bytes": 2 * a * (m * k + m * n) + 2 * n * k * _BYTES[case["weight"]], "flops": 6 * m * n * k}
    sizes = [int(x) for x in case["sizes"].split(",")]
    n = sum(sizes)
    pg = n * (2 * _BYTES[case["param"]] + _BYTES[case["grad"]])
    if case["op"] == "adamw32":
        return {"bytes": pg + 16 * n, "flops": 16 * n}
    # codes of both moments read and written, the values they stand for written, two maxima per block
    # read and written
    return {"bytes": pg + 4 * n + 8 * n + 16 * sum(_blocks(sizes)), "flops": 16 * n}


# ----------------------------------------------------------------------------------------------- inputs

def _generator(seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(int(seed))
    return g


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device=DEVICE, dtype=torch.float32)


def prepare(case, seed):
    g = _generator(seed)
    if case["op"] in ("linear", "train"):
        m, n, k = case["tokens"], case["n"], case["k"]
        x = _normal(g, m, k)
        # a few channels carry activations an order of magnitude larger than the rest
        x[:, torch.randint(0, k, (max(1, k // 256),), generator=g, device=DEVICE)] *= 20.0
        x = x.to(_DTYPE[case["act"]])
        w = _normal(g, n, k) * 0.02
        if case["op"] == "linear":
            codes, scales = _pack_tiles(w.to(torch.bfloat16).float())
            return dict(op="linear", x=x, codes=codes, scales=scales)
        w = w.to(_DTYPE[case["weight"]])
        dy = (_normal(g, m, n) * 1e-3).to(_DTYPE[case["act"]])
        return dict(op="train", x=x.requires_grad_(), w=w.requires_grad_(), dy=dy)
    # The tensors lie in flat buffers, each from a multiple of 2048 on (zeros behind its end), as an
    # optimizer lays out its state; ``tensors`` are the views that it steps.
    sizes = [int(v) for v in case["sizes"].split(",")]
    nb = _blocks(sizes)
    total = sum(nb) * BLOCK
    first = np.concatenate([[0], np.cumsum(nb)])[:-1] * BLOCK
    live = torch.zeros(total, dtype=torch.bool, device=DEVICE)
    for o, n in zip(first, sizes):
        live[o:o + n] = True
    p = (_normal(g, total) * 0.02 * live).to(_DTYPE[case["param"]])
    # gradients and moments vary in size from block to block by a factor of up to ten either way
    size = 10.0 ** (2 * torch.rand(sum(nb), 1, generator=g, device=DEVICE) - 1)
    spread = 1e-3 * size.expand(-1, BLOCK).reshape(-1) * live
    grad = _normal(g, total) * spread
    far = torch.randint(0, total, (max(1, total // 10000),), generator=g, device=DEVICE)
    grad[far] *= 1000.0  # rare large entries
    grad = grad.to(_DTYPE[case["grad"]])
    m = _normal(g, total) * spread * 0.3
    v = (_normal(g, total).square() * 0.2 + 0.8) * spread.square()
    state = dict(op=case["op"], p=p, g=grad, m=m, v=v,
                 scale=torch.full((1,), 0.37, device=DEVICE) if case["clip"] else None)
    views = [(slice(o, o + n), slice(o // BLOCK, o // BLOCK + b)) for o, n, b in zip(first, sizes, nb)]
    if case["op"] == "adamw32":
        state["tensors"] = [(p[a], grad[a], m[a], v[a]) for a, _ in views]
        return state
    cm, am = _quantize(m, True)
    cv, av = _quantize(v, False)
    # the moments' values, written by every pass
    state.update(cm=cm, am=am, cv=cv, av=av, m=torch.empty_like(m), v=torch.empty_like(v))
    state["tensors"] = [(p[a], grad[a], cm[a], cv[a], am[b], av[b]) for a, b in views]
    return state


# --------------------------------------------------------------------------- plain forms: 8-bit products

def _exponents(amax):
    """Least e with amax <= 448 * 2^e (448 = 0.875 * 2^9), at least -127, 0 where amax is 0."""
    f, e = torch.frexp(amax)
    e = e - 9 + (f > 0.875)
    return torch.where(amax > 0, e.clamp(min=-127), torch.zeros_like(e))


def _pad(x, *multiples):
    """Zeros behind the last two axes up to multiples of the given numbers."""
    r, c = (-(-s // q) * q for s, q in zip(x.shape, multiples))
    return torch.nn.functional.pad(x, (0, c - x.shape[1], 0, r - x.shape[0]))


def _e4m3(x, e):
    return (x * torch.exp2(-e.float())).to(torch.float8_e4m3fn)


def _round_rows(x):
    """The values that blocks of 128 along the rows of x stand for, padded to whole blocks."""
    b = _pad(x, 1, KBLOCK)
    b = b.view(x.shape[0], -1, KBLOCK)
    e = _exponents(b.abs().amax(2, keepdim=True))
    return (_e4m3(b, e).float() * torch.exp2(e.float())).view(x.shape[0], -1)


def _tiles(w):
    b = _pad(w, KBLOCK, KBLOCK)
    b = b.view(b.shape[0] // KBLOCK, KBLOCK, b.shape[1] // KBLOCK, KBLOCK)
    e = _exponents(b.abs().amax((1, 3), keepdim=True))
    return _e4m3(b, e), e


def _round_tiles(w):
    """The values that tiles of 128 x 128 of w stand for."""
    codes, e = _tiles(w)
    values = codes.float() * torch.exp2(e.float())
    return values.view(values.shape[0] * KBLOCK, -1)[:w.shape[0], :w.shape[1]]


def _pack_tiles(w):
    """A weight as a server keeps it: e4m3 codes [n, k up to a multiple of 128] and one byte e + 127 per
    tile [ceil(n / 128), ceil(k / 128)]."""
    codes, e = _tiles(w)
    codes = codes.view(codes.shape[0] * KBLOCK, -1)[:w.shape[0]].contiguous()
    return codes, (e + 127).to(torch.uint8).view(e.shape[0], e.shape[2])


def _linear_plain(s):
    x, codes, scales = s["x"], s["codes"], s["scales"]
    scale = torch.exp2(scales.float() - 127.0).repeat_interleave(KBLOCK, 0)[:codes.shape[0]]
    w = codes.float() * scale.repeat_interleave(KBLOCK, 1)
    return (_round_rows(x.float()) @ w.t()).to(x.dtype)


def _train_plain(s):
    with torch.no_grad():
        x, w, dy = s["x"].float(), s["w"].float(), s["dy"].float()
        k = x.shape[1]
        wq = _round_tiles(w)
        y = _round_rows(x)[:, :k] @ wq.t()
        dx = _round_rows(dy)[:, :dy.shape[1]] @ wq
        dw = _round_rows(dy.t().contiguous()) @ _round_rows(x.t().contiguous()).t()
        return [y.to(s["x"].dtype), dx.to(s["x"].dtype), dw.to(s["w"].dtype)]


# -------------------------------------------------------------------------------- plain forms: AdamW steps

def _magnitudes(bits):
    """Values of the dynamic-tree code's patterns of so many bits: e leading zeros, an indicator 1, f
    fraction bits of value j stand for 10^-e (0.1 + 0.9 (j + 1) / 2^f); the pattern 0 for 0."""
    def value(pattern):
        f = pattern.bit_length() - 1
        j = pattern - (1 << f)
        return float(Fraction(1, 10 ** (bits - 1 - f)) * (Fraction(1, 10) + Fraction(9 * (j + 1), 10 << f)))

    return torch.tensor([0.0] + [value(q) for q in range(1, 1 << bits)], dtype=torch.float64).float()


_tables = {}


def _table(signed):
    """Ascending magnitudes on the GPU."""
    if signed not in _tables:
        _tables[signed] = _magnitudes(7 if signed else 8).to(DEVICE)
    return _tables[signed]


def _quantize(x, signed):
    """uint8 codes and block maxima of a flat tensor of whole blocks."""
    t = _table(signed)
    b = x.view(-1, BLOCK)
    amax = b.abs().amax(1, keepdim=True)
    ok = amax >= torch.finfo(torch.float32).tiny
    r = torch.where(ok, 1.0 / amax, torch.zeros_like(amax))
    a = b.abs() * r
    hi = torch.bucketize(a, t).clamp(1, t.numel() - 1)
    code = torch.where(a - t[hi - 1] <= t[hi] - a, hi - 1, hi)
    if signed:
        code = code + 128 * ((b < 0) & ok)
    return code.to(torch.uint8).view(-1), torch.where(ok, amax, torch.zeros_like(amax)).view(-1)


def _values(codes, amax, signed):
    t = _table(signed)
    t = torch.cat([t, -t]) if signed else t
    return (t[codes.long()].view(-1, BLOCK) * amax.view(-1, 1)).view(-1)


def _scalars():
    """Hyper-parameters as binary32 values, and the step's two bias-corrected scalars, rounded once."""
    f = {k: float(np.float32(v)) for k, v in HP.items() if k != "step"}
    t = HP["step"]
    return dict(b1=f["beta1"], b2=f["beta2"], eps=f["eps"], omb1=1.0 - f["beta1"], omb2=1.0 - f["beta2"],
                decay=float(np.float32(1.0 - f["lr"] * f["weight_decay"])),
                step_size=float(np.float32(f["lr"] / (1.0 - f["beta1"] ** t))),
                inv=float(np.float32(1.0 / math.sqrt(1.0 - f["beta2"] ** t))))


def _update_plain(s, m, v):
    c = _scalars()
    g = s["g"].float()
    if s["scale"] is not None:
        g = g * s["scale"]
    m = m * c["b1"] + g * c["omb1"]
    v = v * c["b2"] + (g * g) * c["omb2"]
    u = m / (torch.sqrt(v) * c["inv"] + c["eps"])
    p = s["p"].float() * c["decay"] - u * c["step_size"]
    s["p"].copy_(p)
    return m, v


def _adamw8_plain(s):
    m, v = _update_plain(s, _values(s["cm"], s["am"], True), _values(s["cv"], s["av"], False))
    (cm, am), (cv, av) = _quantize(m, True), _quantize(v, False)
    s["cm"].copy_(cm), s["am"].copy_(am), s["cv"].copy_(cv), s["av"].copy_(av)
    s["m"].copy_(_values(cm, am, True)), s["v"].copy_(_values(cv, av, False))
    return [s["p"], s["m"], s["v"], s["am"], s["av"]]


def _adamw32_plain(s):
    m, v = _update_plain(s, s["m"], s["v"])
    s["m"].copy_(m), s["v"].copy_(v)
    return [s["p"], s["m"], s["v"]]


# --------------------------------------------------------------------------------------------------- run

def run(state):
    op = state["op"]
    if not own:
        return {"linear": _linear_plain, "train": _train_plain, "adamw8": _adamw8_plain,
                "adamw32": _adamw32_plain}[op](state)
    import block_wise_bit_adam8bit_amd as q
    if op == "linear":
        return q.qopt_fp8_linear(state["x"], state["codes"], state["scales"])
    if op == "train":
        y = q.fp8_linear(state["x"], state["w"])
        dx, dw = torch.autograd.grad(y, (state["x"], state["w"]), state["dy"])
        return [y, dx, dw]
    if op == "adamw32":
        if "plan" not in state:  # made once for the tensors that a program steps
            state["plan"] = q.qopt_adamw32bit_plan(state["tensors"])
        q.qopt_adamw32bit_step(state["plan"], grad_scale=state["scale"], **HP)
        return [state["p"], state["m"], state["v"]]
    if "plan" not in state:
        state["plan"] = q.qopt_adamw8bit_plan(state["tensors"])
    q.qopt_adamw8bit_step(state["plan"], grad_scale=state["scale"], **HP)
    # the values that the new codes stand for
    q.qopt_dequantize_blockwise(state["cm"], state["am"], q.SIGNED, out=state["m"])
    q.qopt_dequantize_blockwise(state["cv"], state["av"], q.UNSIGNED, out=state["v"])
    return [state["p"], state["m"], state["v"], state["am"], state["av"]]


# ------------------------------------------------------------------------------------------------- exact

def _exact_round(x, dims):
    """x in binary64, split by ``dims`` (rows, columns of a block), each block as its codes and scale
    stand for it."""
    r, c = dims
    pr, pc = -x.shape[0] % r, -x.shape[1] % c
    z = x.new_zeros(x.shape[0] + pr, x.shape[1] + pc)
    z[:x.shape[0], :x.shape[1]] = x
    z = z.reshape(z.shape[0] // r, r, z.shape[1] // c, c)
    big = z.abs().amax(3).amax(1)[:, None, :, None]
    e = torch.ceil(torch.log2(torch.where(big > 0, big, torch.ones_like(big)) / 448.0))
    e = e - (448.0 * torch.exp2(e - 1) >= big).double()  # log2 is rounded: put e right by comparison
    e = e + (448.0 * torch.exp2(e) < big).double()
    scale = torch.exp2(torch.where(big > 0, e.clamp(min=-127), torch.zeros_like(e)))
    y = z / scale
    grid = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    y = torch.round(y / grid) * grid * scale
    return y.reshape(x.shape[0] + pr, x.shape[1] + pc)[:x.shape[0], :x.shape[1]]


def exact(case, seed):
    s = prepare(case, seed)
    with torch.no_grad():
        if case["op"] == "linear":
            n, k = case["n"], case["k"]
            up = lambda e: torch.exp2(s["scales"].double() - 127)[  # noqa: E731
                (torch.arange(n, device=DEVICE) // KBLOCK)[:, None],
                (torch.arange(k, device=DEVICE) // KBLOCK)[None, :]]
            w = s["codes"][:, :k].float().double() * up(None)
            return _exact_round(s["x"].double(), (1, KBLOCK)) @ w.t()
        if case["op"] == "train":
            x, w, dy = s["x"].double(), s["w"].double(), s["dy"].double()
            wq = _exact_round(w, (KBLOCK, KBLOCK))
            return [_exact_round(x, (1, KBLOCK)) @ wq.t(), _exact_round(dy, (1, KBLOCK)) @ wq,
                    _exact_round(dy, (KBLOCK, 1)).t() @ _exact_round(x, (KBLOCK, 1))]
        lr, b1, b2, eps, wd = (float(np.float32(HP[k])) for k in ("lr", "beta1", "beta2", "eps", "weight_decay"))
        t = HP["step"]
        g = s["g"].double() * (s["scale"].double() if s["scale"] is not None else 1.0)
        if case["op"] == "adamw32":
            m, v = s["m"].double(), s["v"].double()
        else:
            tree = torch.tensor([float(a) for a in _magnitudes(7)], dtype=torch.float64, device=DEVICE)
            flat = torch.tensor([float(a) for a in _magnitudes(8)], dtype=torch.float64, device=DEVICE)
            cm = s["cm"].long()
            m = tree[cm % 128] * (1 - 2 * (cm // 128)) * s["am"].double().repeat_interleave(BLOCK)
            v = flat[s["cv"].long()] * s["av"].double().repeat_interleave(BLOCK)
        m = b1 * m + (1 - b1) * g
        v = b2 * v + (1 - b2) * g ** 2
        p = s["p"].double() * (1 - lr * wd)
        p = p - lr * (m / (1 - b1 ** t)) / ((v / (1 - b2 ** t)).sqrt() + eps)
        if case["op"] == "adamw32":
            return [p, m, v]
        # The new codes depend on the binary32 rounding of values next to a border between two codes, so
        # the values that they stand for have no counterpart in 64 bits; the block maxima have.
        return [p, None, None, m.view(-1, BLOCK).abs().amax(1), v.view(-1, BLOCK).amax(1)]
