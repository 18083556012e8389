"""Operators next to the 8-bit ones, as cases that can be timed and compared: what a feed-forward block takes
before, in and after its products.

* ``norm``: layer normalisation over the last axis, forward alone (``train`` false) or with the gradients of the
  input, the weight and the bias.
* ``quantize``: microscaled 4-bit floating point (e2m1 codes, one power-of-two scale per block of 32), written
  and read back.
* ``linear``: the product of activations, quantized on the way, with a weight held in that format, as a server
  calls it; with ``train`` the differentiable layer, whose forward pass is that product of a full-precision
  weight and whose gradients are the 8-bit products of the same layer.
* ``orthogonalize``: five Newton-Schulz iterations on matrices divided by their Frobenius norm.
* ``muon``: one optimizer step over many matrices: momentum (in 8-bit codes or in binary32), the orthogonalised
  update, decoupled weight decay.

``run`` computes the plain form with elementary torch operations, or, where ``own`` is true, makes the calls of
this repository's package.  ``exact`` computes the same results in binary64, written apart.

Definitions.  Layer normalisation: y = (x - mean) / sqrt(var + eps) * w + b, var the mean of (x - mean)^2.

4 bits: a block of 32 consecutive values x of a row has e = the least integer with max|x| <= 6 * 2^e, at least
-127 (0 for a block of zeros); it stores e + 127 in a byte and each x * 2^-e rounded to e2m1 (0, 0.5, 1, 1.5, 2,
3, 4, 6 and their negatives), nearest, ties to the even code.  8 bits: blocks of 128 along the summed axis (tiles
of 128 x 128 for the weight), 448 instead of 6, e4m3.

A matrix in 4 bits is kept as codes, uint8 [rows, K / 2] with the value of the even column in the low half of a
byte, K the columns rounded up to a multiple of 256, and scales, uint8 [K / 128, R, 4], R the rows rounded up to a
multiple of 16: scales[i, r, j] belongs to columns 128 i + 32 j to 128 i + 32 j + 31 of row r.

Newton-Schulz: X = U / max(|U|, 1e-7) and five times X = a X + (b A + c A^2) X with A = X X^T, a, b, c = 3.4445,
-4.775, 2.0315; U is taken transposed where it has more rows than columns.

Muon, for a gradient g scaled by s, hyper-parameters in binary32:
    m = mu m + (1 - mu) g s      u = mu m + (1 - mu) g s
    p = p (1 - lr wd) - lr 0.2 sqrt(max(rows, columns)) NewtonSchulz(u)
with 8-bit state m is then requantized in blocks of 2048 (nearest code of the magnitude over the block's largest).
"""

import math
from fractions import Fraction

import numpy as np
import torch

own = False

BLOCK = 2048  # values per block of the 8-bit optimizer state
DEVICE = "cuda"

HP = dict(lr=2e-3, momentum=0.95, weight_decay=0.1)
EPS_NORM, EPS_MUON = 1e-5, 1e-7
NS = (3.4445, -4.775, 2.0315)
STEPS = 5


# ------------------------------------------------------------------------------------------------ cases

_GPT_BLOCK = "2048x2048,2048x2048,2048x2048,2048x2048,8192x2048,2048x8192"


def listed():
    return [
        # one token of the 7B set's width in front of a projection: latency
        dict(name="norm one token 4096", op="norm", tokens=1, dim=4096, act="bf16", weight="f32", train=False),
        # a ragged batch at the 1.3B set's width, everything in fp32
        dict(name="norm train 1999x2048 f32", op="norm", tokens=1999, dim=2048, act="f32", weight="f32", train=True),
        # the largest: the 7B set's width, a batch of 65536 tokens
        dict(name="norm train 65536x4096 bf16", op="norm", tokens=65536, dim=4096, act="bf16", weight="f32",
             train=True),
        # packing the 7B set's gate projection for serving
        dict(name="quantize 11008x4096 bf16", op="quantize", rows=11008, cols=4096, act="bf16"),
        # an odd matrix in fp32
        dict(name="quantize 777x1000 f32", op="quantize", rows=777, cols=1000, act="f32"),
        # one token through an attention projection of the 7B set: latency and the weight's bytes
        dict(name="linear one token 4096x4096", op="linear", tokens=1, n=4096, k=4096, act="bf16", train=False),
        # the largest product served: 8192 tokens of prompts through the 7B set's gate projection
        dict(name="linear 8192 tokens 11008x4096", op="linear", tokens=8192, n=11008, k=4096, act="bf16",
             train=False),
        # training towards a 4-bit weight: a ragged batch through the 1.3B set's second feed-forward product
        dict(name="linear train 1999x2048x8192", op="linear", tokens=1999, n=2048, k=8192, act="bf16",
             weight="f32", train=True),
        # the update of one small odd matrix: latency
        dict(name="orthogonalize 99x300 f32", op="orthogonalize", batch=1, rows=99, cols=300, act="f32"),
        # the 1.3B set's attention projections of one block
        dict(name="orthogonalize 4x2048x2048 bf16", op="orthogonalize", batch=4, rows=2048, cols=2048, act="bf16"),
        # every matrix of one block of the 1.3B set, 8-bit momentum, bf16 parameters, gradients clipped
        dict(name="muon 8-bit 1.3B block bf16", op="muon", shapes=_GPT_BLOCK, bits=8, param="bf16", grad="bf16",
             clip=True),
        # the 7B set's down projection, fp32 master weights and momentum: wide, the largest
        dict(name="muon 32-bit 4096x11008", op="muon", shapes="4096x11008", bits=32, param="f32", grad="bf16",
             clip=False),
    ]


def draw(rng):
    def spread(lo, hi):
        return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    op = rng.choice(["norm", "norm", "quantize", "linear", "linear", "orthogonalize", "muon"])
    act = rng.choice(["bf16", "bf16", "f32"])
    if op == "norm":
        dim = spread(16, 16384)
        return dict(op=op, tokens=min(spread(1, 65536), 65536 * 4096 // dim), dim=dim, act=act,
                    weight=rng.choice(["f32", "f32", "bf16"]), train=rng.random() < 0.7)
    if op == "quantize":
        return dict(op=op, rows=spread(1, 11008), cols=spread(1, 8192), act=act)
    if op == "linear":
        n, k, train = spread(16, 11008), spread(16, 8192), rng.random() < 0.4
        most = (1999 * 2048 * 8192 if train else 8192 * 11008 * 4096) // (n * k)
        case = dict(op=op, tokens=min(most, spread(1, 8192)), n=n, k=k, act=act, train=train)
        if train:
            case["weight"] = rng.choice(["bf16", "f32"])
        return case
    if op == "orthogonalize":
        rows, cols = spread(1, 4096), spread(1, 4096)
        cost = min(rows, cols) ** 2 * max(rows, cols)
        return dict(op=op, batch=min(spread(1, 16), max(1, 4 * 2048 ** 3 // cost)), rows=rows, cols=cols, act=act)
    shapes, left = [], 4096 * 4096 * 11008
    for _ in range(spread(1, 12)):
        rows, cols = spread(2, 4096), spread(2, 4096)
        cost = min(rows, cols) ** 2 * max(rows, cols)
        if cost <= left:
            shapes += ["%dx%d" % (rows, cols)] * rng.choice([1, 1, 2])
            left -= cost * 2
    return dict(op=op, shapes=",".join(shapes or ["64x64"]), bits=rng.choice([8, 32]),
                param=rng.choice(["f32", "bf16"]), grad=rng.choice(["f32", "bf16"]), clip=rng.random() < 0.5)


_DTYPE = {"f32": torch.float32, "bf16": torch.bfloat16}
_BYTES = {"f32": 4, "bf16": 2}


def _shapes(case):
    return [tuple(int(v) for v in s.split("x")) for s in case["shapes"].split(",")]


def _blocks(n):
    return -(-n // BLOCK)


def _ns_flops(rows, cols):
    """The iterations' products, the symmetric ones counted by half.  In units of 2 m^3 (m <= n): five times
    A, A^2 and the product with X take 7.5 n / m + 2.5; with the iterations carried out on A = X X^T alone, and
    their polynomials applied to X after the third and the fifth, 3 n / m + 7."""
    m, n = sorted((rows, cols))
    return 2.0 * m ** 3 * min(7.5 * n / m + 2.5, 3 * n / m + 7)


def work(case):
    a = _BYTES[case["act"]] if "act" in case else 0
    if case["op"] == "norm":
        n, d, w = case["tokens"], case["dim"], _BYTES[case["weight"]]
        # x and y; with gradients x, dy in and y, dx, dw, db out
        return {"bytes": (4 if case["train"] else 2) * n * d * a + (4 if case["train"] else 2) * d * w,
                "flops": (20 if case["train"] else 8) * n * d}
    if case["op"] == "quantize":
        n = case["rows"] * case["cols"]
        return {"bytes": n * (2 * a + 17 / 32), "flops": 4 * n}
    if case["op"] == "linear":
        m, n, k = case["tokens"], case["n"], case["k"]
        if not case["train"]:
            return {"bytes": (m * k + m * n) * a + n * k * 17 / 32, "flops": 2 * m * n * k}
        return {"bytes": 2 * a * (m * k + m * n) + 2 * n * k * _BYTES[case["weight"]], "flops": 6 * m * n * k}
    if case["op"] == "orthogonalize":
        b, r, c = case["batch"], case["rows"], case["cols"]
        return {"bytes": 2 * b * r * c * a, "flops": b * _ns_flops(r, c)}
    # p and m read and written, g read; with codes, the values that they stand for written too
    n = sum(r * c for r, c in _shapes(case))
    state = 8 if case["bits"] == 32 else 6 + 8 / BLOCK
    return {"bytes": n * (2 * _BYTES[case["param"]] + _BYTES[case["grad"]] + state),
            "flops": sum(_ns_flops(r, c) for r, c in _shapes(case))}


# ----------------------------------------------------------------------------------------------- inputs

def _generator(seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(int(seed))
    return g


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device=DEVICE, dtype=torch.float32)


def _gradients(g, *shape):
    """Gradients of a matrix: a few directions that most of it lies in, noise, and rare large entries."""
    *batch, rows, cols = shape
    x = _normal(g, *shape) * 1e-3
    r = min(8, rows, cols)
    big = _normal(g, *batch, rows, r) @ _normal(g, *batch, cols, r).transpose(-1, -2).contiguous()
    x += big * (2e-3 / math.sqrt(r))
    n = x.numel()
    x.view(-1)[torch.randint(0, n, (max(1, n // 10000),), generator=g, device=DEVICE)] *= 10.0
    return x


def prepare(case, seed):
    g = _generator(seed)
    op = case["op"]
    if op == "norm":
        n, d = case["tokens"], case["dim"]
        x = _normal(g, n, d) + 0.1 * _normal(g, n, 1)
        # a few channels carry activations an order of magnitude larger than the rest
        x[:, torch.randint(0, d, (max(1, d // 256),), generator=g, device=DEVICE)] *= 20.0
        w = (1.0 + 0.1 * _normal(g, d)).to(_DTYPE[case["weight"]])
        b = (0.1 * _normal(g, d)).to(_DTYPE[case["weight"]])
        s = dict(op=op, train=case["train"], x=x.to(_DTYPE[case["act"]]), w=w, b=b)
        if case["train"]:
            s["dy"] = (_normal(g, n, d) * 1e-3).to(_DTYPE[case["act"]])
            for k in ("x", "w", "b"):
                s[k].requires_grad_()
        return s
    if op == "quantize":
        x = _normal(g, case["rows"], case["cols"]) * 0.02
        far = torch.randint(0, x.numel(), (max(1, x.numel() // 10000),), generator=g, device=DEVICE)
        x.view(-1)[far] *= 50.0
        x[case["rows"] // 2:case["rows"] // 2 + 1] = 0.0  # a row that is all padding
        return dict(op=op, x=x.to(_DTYPE[case["act"]]))
    if op == "linear":
        m, n, k = case["tokens"], case["n"], case["k"]
        x = _normal(g, m, k)
        x[:, torch.randint(0, k, (max(1, k // 256),), generator=g, device=DEVICE)] *= 20.0
        x = x.to(_DTYPE[case["act"]])
        w = _normal(g, n, k) * 0.02
        if not case["train"]:
            codes, scales = _pack(w.to(torch.bfloat16).float())
            return dict(op=op, train=False, x=x, codes=codes, scales=scales)
        dy = (_normal(g, m, n) * 1e-3).to(_DTYPE[case["act"]])
        return dict(op=op, train=True, x=x.requires_grad_(), w=w.to(_DTYPE[case["weight"]]).requires_grad_(), dy=dy)
    if op == "orthogonalize":
        return dict(op=op, x=_gradients(g, case["batch"], case["rows"], case["cols"]).to(_DTYPE[case["act"]]))
    state = dict(op=op, bits=case["bits"], tensors=[], values=[],
                 scale=torch.full((1,), 0.37, device=DEVICE) if case["clip"] else None)
    for rows, cols in _shapes(case):
        p = (_normal(g, rows, cols) * 0.02).to(_DTYPE[case["param"]])
        grad = _gradients(g, rows, cols).to(_DTYPE[case["grad"]])
        m = _gradients(g, rows, cols) * 0.3
        if case["bits"] == 8:
            codes, amax = _quantize8(m)
            state["values"].append(torch.empty_like(m))  # what the new codes stand for, written by every pass
            state["tensors"].append((p, grad, codes, amax))
        else:
            state["tensors"].append((p, grad, m))
    return state


# ----------------------------------------------------------------------- plain forms: layer normalisation

def _norm_plain(s):
    with torch.no_grad():
        x, w, b = s["x"].float(), s["w"].float(), s["b"].float()
        c = x - x.mean(1, keepdim=True)
        rstd = 1.0 / torch.sqrt((c * c).mean(1, keepdim=True) + EPS_NORM)
        h = c * rstd
        y = (h * w + b).to(s["x"].dtype)
        if not s["train"]:
            return y
        dy = s["dy"].float()
        dw, db = (dy * h).sum(0), dy.sum(0)
        v = dy * w
        dx = (v - v.mean(1, keepdim=True) - h * (v * h).mean(1, keepdim=True)) * rstd
        return [y, dx.to(s["x"].dtype), dw.to(s["w"].dtype), db.to(s["b"].dtype)]


# -------------------------------------------------------------------------------- plain forms: products

def _exponents(amax, fraction, power):
    """Least e with amax <= fraction * 2^(e + power), fraction in [0.5, 1): at least -127, 0 where amax is 0."""
    f, e = torch.frexp(amax)
    e = e - power + (f > fraction)
    return torch.where(amax > 0, e.clamp(min=-127), torch.zeros_like(e))


def _pad(x, *multiples):
    """Zeros behind the last two axes up to multiples of the given numbers."""
    r, c = (-(-s // q) * q for s, q in zip(x.shape, multiples))
    return torch.nn.functional.pad(x, (0, c - x.shape[1], 0, r - x.shape[0]))


def _blocks4(x):
    """Blocks of 32 along the rows of x, padded to whole ones: e2m1 values [rows, blocks, 32] and exponents."""
    b = _pad(x, 1, 32)
    b = b.view(x.shape[0], -1, 32)
    e = _exponents(b.abs().amax(2, keepdim=True), 0.75, 3)  # 6 = 0.75 * 2^3
    y = b * torch.exp2(-e.float())
    a = y.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    return torch.round(y / step) * step, e


def _round4(x):
    """The values that the 4-bit blocks of x stand for."""
    y, e = _blocks4(x)
    return (y * torch.exp2(e.float())).view(x.shape[0], -1)[:, :x.shape[1]]


def _pack(w):
    """A weight as a server keeps it: codes and scales as laid out above."""
    n, k = w.shape
    y, e = _blocks4(_pad(w, 1, 256))
    grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=w.device)
    code = torch.bucketize(y.abs(), grid) + 8 * (y < 0)
    code = code.view(n, -1, 2).to(torch.uint8)
    scales = torch.full((y.shape[1] // 4, -(-n // 16) * 16, 4), 127, dtype=torch.uint8, device=w.device)
    scales[:, :n] = (e + 127).to(torch.uint8).view(n, -1, 4).transpose(0, 1)
    return (code[:, :, 0] + 16 * code[:, :, 1]).contiguous(), scales


def _unpack(codes, scales):
    """The values of a packed weight, padding included."""
    grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=codes.device)
    grid = torch.cat([grid, -grid])
    n = codes.shape[0]
    y = grid[torch.stack([codes & 15, codes >> 4], 2).long()].view(n, -1, 32)
    return (y * torch.exp2(scales[:, :n].transpose(0, 1).reshape(n, -1, 1).float() - 127.0)).view(n, -1)


def _round8(x, rows):
    """The values that 8-bit blocks of rows x 128 of x stand for."""
    b = _pad(x, rows, 128)
    b = b.view(b.shape[0] // rows, rows, -1, 128)
    e = _exponents(b.abs().amax((1, 3), keepdim=True), 0.875, 9)  # 448 = 0.875 * 2^9
    y = (b * torch.exp2(-e.float())).to(torch.float8_e4m3fn).float() * torch.exp2(e.float())
    return y.view(-1, y.shape[2] * 128)[:x.shape[0], :x.shape[1]]


def _linear_plain(s):
    with torch.no_grad():
        x = s["x"].float()
        if not s["train"]:
            w = _unpack(s["codes"], s["scales"])[:, :x.shape[1]]
            return (_round4(x) @ w.t()).to(s["x"].dtype)
        w, dy = s["w"].float(), s["dy"].float()
        y = _round4(x) @ _round4(w).t()
        dx = _round8(dy, 1) @ _round8(w, 128)
        dw = _round8(dy.t().contiguous(), 1) @ _round8(x.t().contiguous(), 1).t()
        return [y.to(s["x"].dtype), dx.to(s["x"].dtype), dw.to(s["w"].dtype)]


# -------------------------------------------------------------------------------- plain forms: Muon

def _newton_schulz(u):
    """Of matrices [..., m, n] in 32 bits."""
    a, b, c = NS
    norm = u.double().square().sum((-1, -2), keepdim=True).sqrt().clamp(min=EPS_MUON)
    x = (u.double() / norm).float()
    tall = x.shape[-2] > x.shape[-1]
    if tall:
        x = x.transpose(-1, -2).contiguous()
    for _ in range(STEPS):
        g = x @ x.transpose(-1, -2).contiguous()
        x = a * x + (b * g + c * (g @ g)) @ x
    return x.transpose(-1, -2) if tall else x


def _magnitudes(bits):
    """Values of the dynamic-tree code's patterns of so many bits: e leading zeros, an indicator 1, f
    fraction bits of value j stand for 10^-e (0.1 + 0.9 (j + 1) / 2^f); the pattern 0 for 0."""
    def value(pattern):
        f = pattern.bit_length() - 1
        j = pattern - (1 << f)
        return float(Fraction(1, 10 ** (bits - 1 - f)) * (Fraction(1, 10) + Fraction(9 * (j + 1), 10 << f)))

    return torch.tensor([0.0] + [value(q) for q in range(1, 1 << bits)], dtype=torch.float64)


_tables = {}


def _table():
    """Ascending magnitudes of the signed code, on the GPU."""
    if "signed" not in _tables:
        _tables["signed"] = _magnitudes(7).float().to(DEVICE)
    return _tables["signed"]


def _by_blocks(x):
    x = x.reshape(-1)
    return torch.nn.functional.pad(x, (0, -x.numel() % BLOCK)).view(-1, BLOCK)


def _quantize8(x):
    """uint8 codes of x's shape and block maxima."""
    t = _table()
    b = _by_blocks(x)
    amax = b.abs().amax(1, keepdim=True)
    ok = amax >= torch.finfo(torch.float32).tiny
    r = torch.where(ok, 1.0 / amax, torch.zeros_like(amax))
    a = b.abs() * r
    hi = torch.bucketize(a, t).clamp(1, t.numel() - 1)
    code = torch.where(a - t[hi - 1] <= t[hi] - a, hi - 1, hi) + 128 * ((b < 0) & ok)
    code = code.to(torch.uint8).view(-1)[:x.numel()].view(x.shape)
    return code, torch.where(ok, amax, torch.zeros_like(amax)).view(-1)


def _values8(codes, amax):
    t = _table()
    y = torch.cat([t, -t])[_by_blocks(codes).long()] * amax.view(-1, 1)
    return y.view(-1)[:codes.numel()].view(codes.shape)


def _f32(x):
    return float(np.float32(x))


def _muon_plain(s):
    mu, lr, wd = (_f32(HP[k]) for k in ("momentum", "lr", "weight_decay"))
    out = []
    for i, (p, grad, m, *amax) in enumerate(s["tensors"]):
        g = grad.float()
        if s["scale"] is not None:
            g = g * s["scale"]
        old = _values8(m, amax[0]) if amax else m
        new = old * mu + g * (1.0 - mu)
        u = new * mu + g * (1.0 - mu)
        rate = lr * 0.2 * math.sqrt(max(p.shape))
        p.copy_(p.float() * (1.0 - lr * wd) - _newton_schulz(u) * rate)
        if amax:
            codes, top = _quantize8(new)
            m.copy_(codes), amax[0].copy_(top)
            s["values"][i].copy_(_values8(m, amax[0]))
            out += [p, s["values"][i], amax[0]]
        else:
            m.copy_(new)
            out += [p, m]
    return out


# --------------------------------------------------------------------------------------------------- run

def run(state):
    op = state["op"]
    if not own:
        if op == "quantize":
            return _round4(state["x"].float()).to(state["x"].dtype)
        if op == "orthogonalize":
            return _newton_schulz(state["x"].float()).to(state["x"].dtype).contiguous()
        return {"norm": _norm_plain, "linear": _linear_plain, "muon": _muon_plain}[op](state)
    import block_wise_bit_adam8bit_amd as q
    if op == "norm":
        if not state["train"]:
            return q.qopt_layer_norm_forward(state["x"], state["w"], state["b"], EPS_NORM, save_stats=False)[0]
        y = q.layer_norm(state["x"], state["w"], state["b"], EPS_NORM)
        return [y, *torch.autograd.grad(y, (state["x"], state["w"], state["b"]), state["dy"])]
    if op == "quantize":
        codes, scales = q.qopt_fp4_quantize(state["x"])
        return q.qopt_fp4_dequantize(codes, scales, state["x"].shape[1], state["x"].dtype)
    if op == "linear":
        if not state["train"]:
            return q.qopt_fp4_linear(state["x"], state["codes"], state["scales"])
        y = q.fp4_linear(state["x"], state["w"])
        return [y, *torch.autograd.grad(y, (state["x"], state["w"]), state["dy"])]
    if op == "orthogonalize":
        return q.qopt_orthogonalize(state["x"], steps=STEPS, eps=EPS_MUON)
    if "plan" not in state:  # made once for the tensors that a program steps
        state["plan"] = (q.qopt_muon8bit_plan if state["bits"] == 8 else q.qopt_muon32bit_plan)(state["tensors"])
    step = q.qopt_muon8bit_step if state["bits"] == 8 else q.qopt_muon32bit_step
    step(state["plan"], lr=HP["lr"], momentum=HP["momentum"], weight_decay=HP["weight_decay"], nesterov=True,
         adjust="match_rms_adamw", steps=STEPS, eps=EPS_MUON, grad_scale=state["scale"])
    if state["bits"] == 32:
        return [x for p, _, m in state["tensors"] for x in (p, m)]
    out = []
    for (p, _, codes, amax), values in zip(state["tensors"], state["values"]):
        q.qopt_dequantize_blockwise(codes, amax, q.SIGNED, out=values)  # the values that the new codes stand for
        out += [p, values, amax]
    return out


# ------------------------------------------------------------------------------------------------- exact

def _scale64(big, top):
    """2^e, e the least integer with big <= top * 2^e, at least -127; 1 where big is 0."""
    e = torch.ceil(torch.log2(torch.where(big > 0, big, torch.ones_like(big)) / top))
    e = e - (top * torch.exp2(e - 1) >= big).double()  # log2 is rounded: put e right by comparison
    e = e + (top * torch.exp2(e) < big).double()
    return torch.exp2(torch.where(big > 0, e.clamp(min=-127), torch.zeros_like(e)))


def _exact4(x):
    """x in binary64 as its 4-bit blocks stand for it: the nearest of the sixteen values, the even of two."""
    rows, cols = x.shape
    z = x.new_zeros(rows, -(-cols // 32) * 32)
    z[:, :cols] = x
    z = z.reshape(rows, -1, 32)
    scale = _scale64(z.abs().amax(2, keepdim=True), 6.0)
    a = z.abs() / scale
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=x.device)
    mid = (grid[1:] + grid[:-1]) / 2
    code = torch.bucketize(a, mid)  # a border itself goes to the code below it
    code = code + ((code < 7) & (code % 2 == 1) & (a == mid[code.clamp(max=6)])).long()
    y = grid[code] * torch.sign(z) * scale
    return y.reshape(rows, -1)[:, :cols]


def _exact8(x, dims):
    """x in binary64, split by ``dims`` (rows, columns of a block), each block as its e4m3 codes and scale
    stand for it."""
    r, c = dims
    pr, pc = -x.shape[0] % r, -x.shape[1] % c
    z = x.new_zeros(x.shape[0] + pr, x.shape[1] + pc)
    z[:x.shape[0], :x.shape[1]] = x
    z = z.reshape(z.shape[0] // r, r, z.shape[1] // c, c)
    scale = _scale64(z.abs().amax(3).amax(1)[:, None, :, None], 448.0)
    y = z / scale
    grid = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    y = torch.round(y / grid) * grid * scale
    return y.reshape(x.shape[0] + pr, x.shape[1] + pc)[:x.shape[0], :x.shape[1]]


def _exact_norm(s):
    x, w, b = s["x"].double(), s["w"].double(), s["b"].double()
    var, mean = torch.var_mean(x, 1, unbiased=False, keepdim=True)
    y = (x - mean) * (var + EPS_NORM).rsqrt() * w + b
    if not s["train"]:
        return y
    std = (var + EPS_NORM).sqrt()
    dy, h = s["dy"].double(), (x - mean) / std
    d = x.shape[1]
    v = dy * w
    dx = (d * v - v.sum(1, keepdim=True) - h * (v * h).sum(1, keepdim=True)) / (d * std)
    return [y, dx, (dy * h).sum(0), dy.sum(0)]


def _exact_ns(u):
    """The odd polynomial a s + b s^3 + c s^5 five times over, on the matrix itself."""
    x = u / u.square().sum((-1, -2), keepdim=True).sqrt().clamp(min=EPS_MUON)
    for _ in range(STEPS):
        if x.shape[-2] <= x.shape[-1]:
            y = x @ x.transpose(-1, -2).contiguous()
            x = NS[0] * x + NS[1] * (y @ x) + NS[2] * (y @ (y @ x))
        else:
            y = x.transpose(-1, -2).contiguous() @ x
            x = NS[0] * x + NS[1] * (x @ y) + NS[2] * ((x @ y) @ y)
    return x


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    with torch.no_grad():
        if op == "norm":
            return _exact_norm(s)
        if op == "quantize":
            return _exact4(s["x"].double())
        if op == "linear":
            n, k = case["n"], case["k"]
            if not case["train"]:
                sign = 1.0 - 2.0 * (torch.arange(16, device=DEVICE) // 8).double()
                value = torch.tensor([0, 1, 2, 3, 4, 6, 8, 12] * 2, device=DEVICE).double() / 2 * sign
                col = torch.arange(k, device=DEVICE)
                code = (s["codes"][:, col // 2].long() >> (4 * (col % 2))) % 16
                up = s["scales"][col // 128, :, col // 32 % 4].t()[:n].double() - 127
                return _exact4(s["x"].double()) @ (value[code] * torch.exp2(up)).t().contiguous()
            x, w, dy = s["x"].double(), s["w"].double(), s["dy"].double()
            return [_exact4(x) @ _exact4(w).t(), _exact8(dy, (1, 128)) @ _exact8(w, (128, 128)),
                    _exact8(dy, (128, 1)).t() @ _exact8(x, (128, 1))]
        if op == "orthogonalize":
            return _exact_ns(s["x"].double())
        lr, mu, wd = (_f32(HP[k]) for k in ("lr", "momentum", "weight_decay"))
        tree = torch.cat([_magnitudes(7), -_magnitudes(7)]).to(DEVICE)
        out = []
        for p, grad, m, *amax in s["tensors"]:
            g = grad.double() * (s["scale"].double() if s["scale"] is not None else 1.0)
            if amax:
                size = amax[0].double().repeat_interleave(BLOCK)[:m.numel()].view(m.shape)
                m = tree[m.long()] * size
            m = mu * m.double() + (1 - mu) * g
            p = p.double() * (1 - lr * wd) - lr * 0.2 * max(p.shape) ** 0.5 * _exact_ns(mu * m + (1 - mu) * g)
            # the new codes depend on the binary32 rounding of values next to a border between two codes, so
            # the values that they stand for have no counterpart in 64 bits; the block maxima have
            out += [p, None, _by_blocks(m).abs().amax(1)] if amax else [p, m]
        return out
