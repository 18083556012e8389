"""Linear products in 8-bit floating point: wrappers with the C ABI's names
(include/qopt_fp8.h), an autograd function and a torch module.

The block-wise quantization of the 8-bit optimizers summary page (§2 "Block-wise
Quantization") for the products of a linear layer: e4m3 codes with one power-of-two
scale per 128 values along the summed axis (activations, upstream gradients) or per
tile of 128 x 128 (weights).  Every step runs in libqopt's HIP kernels; torch allocates
outputs and workspaces and supplies the current stream.
"""

import ctypes
import math
from typing import NamedTuple

import torch
from torch.autograd import forward_ad
from torch.autograd.function import once_differentiable

from . import _lib
from ._lib import (LIB, QOPT_BF16, QOPT_F32, QOPT_FP8_BLOCK, QOPT_FP8_FEW_ROWS, QOPT_FP8_ROWS,
                   QOPT_FP8_TILES)
from .embedding import qopt_embedding_xavier_init

_DT = {torch.float32: QOPT_F32, torch.bfloat16: QOPT_BF16}
CODE_DTYPE = torch.float8_e4m3fn
_is_tracing = torch._C._is_tracing  # torch.jit.is_tracing takes twice as long


class Fp8Matrix(NamedTuple):
    """A quantized matrix: float8_e4m3fn codes [rows, columns up to a multiple of 128] and
    uint8 scales, each standing for 2^(scale - 127): one per 128 values of a row,
    [columns / 128, rows up to a multiple of 16], or one per tile of 128 x 128,
    [ceil(rows / 128), columns / 128]."""
    codes: torch.Tensor
    scales: torch.Tensor


def _blocks(n):
    return -(-int(n) // QOPT_FP8_BLOCK)


def _check_dtype(dtype, what):
    if dtype not in _DT:
        raise TypeError(f"{what} must be float32 or bfloat16, not {dtype}")
    return _DT[dtype]


def _same_gpu(first, *others):
    index = first.get_device() if first.is_cuda else -1
    if index < 0:
        raise ValueError("all tensors must be on a GPU")
    for t in others:
        if not t.is_cuda:
            raise ValueError("all tensors must be on a GPU")
        if t.get_device() != index:
            raise ValueError("all tensors must be on the same GPU")
    return first.device


def _row_stride(t, what):
    """Elements between the rows of a 2-D tensor whose rows are contiguous."""
    rows, cols = t.shape
    if t.is_contiguous():
        return cols
    far, near = t.stride()
    if cols > 1 and near != 1:
        raise ValueError(f"the rows of {what} must be contiguous")
    if rows <= 1:
        return cols
    if far < cols:
        raise ValueError(f"the rows of {what} must not overlap")
    return far


def _quantized(codes, scales, what):
    """Checks a (codes, scales) pair; returns its form."""
    if codes.dtype is not CODE_DTYPE or scales.dtype is not torch.uint8:
        raise TypeError(f"{what}: codes must be float8_e4m3fn and scales uint8")
    if codes.dim() != 2 or codes.shape[1] % QOPT_FP8_BLOCK:
        raise ValueError(f"{what}: codes must be 2-D with a multiple of {QOPT_FP8_BLOCK} columns")
    rows, kb = codes.shape
    kb //= QOPT_FP8_BLOCK
    if not codes.is_contiguous() or not scales.is_contiguous():
        raise ValueError(f"{what}: codes and scales must be contiguous")
    # the two shapes differ for every matrix with elements: rows <= 16 has 16 columns in the
    # first and one row in the second, more rows have fewer than rows / 16 tiles
    shape, by_rows, by_tiles = scales.shape, (kb, -(-rows // 16) * 16), (-(-rows // QOPT_FP8_BLOCK), kb)
    if shape == by_rows:
        return QOPT_FP8_ROWS
    if shape == by_tiles:
        return QOPT_FP8_TILES
    raise ValueError(f"{what}: scales must be {by_rows} or {by_tiles}, not {tuple(shape)}")


def _empty_matrix(rows, cols, tiles, device):
    kb = _blocks(cols)
    return Fp8Matrix(
        torch.empty(rows, kb * QOPT_FP8_BLOCK, dtype=CODE_DTYPE, device=device),
        torch.empty((_blocks(rows), kb) if tiles else (kb, -(-rows // 16) * 16),
                    dtype=torch.uint8, device=device))


# The launches behind the functions below, for operands that are known to be right.

def _quantize(x, dt, ldx, tiles, normal, transposed):
    rows, cols = x.shape
    dev = x.device
    a = _empty_matrix(rows, cols, tiles, dev) if normal else None
    b = _empty_matrix(cols, rows, tiles, dev) if transposed else None
    if rows and cols:
        _lib.call("qopt_fp8_quantize", dev, x.data_ptr(), dt, rows, cols, ldx,
                  QOPT_FP8_TILES if tiles else QOPT_FP8_ROWS,
                  *((a.codes.data_ptr(), a.scales.data_ptr()) if normal else (None, None)),
                  *((b.codes.data_ptr(), b.scales.data_ptr()) if transposed else (None, None)))
    return a, b


def _sizes(rows, cols, tiles):
    """Bytes of the codes of a quantized matrix, and of both its parts up to a whole page: what
    follows starts on a cache line (codes that straddle them cost a training pass of 8192 x 11008 x
    4096 8 %)."""
    kb = _blocks(cols)
    codes = rows * kb * QOPT_FP8_BLOCK
    scales = _blocks(rows) * kb if tiles else kb * (-(-rows // 16) * 16)
    return codes, -(-(codes + scales) // 4096) * 4096


def _room(query, name, m, n, k, dt):
    need = ctypes.c_size_t(0)
    _lib.check(name, query(m, n, k, dt, ctypes.byref(need)))
    return need.value


def _workspace(query, name, m, n, k, dt, dev):
    """(tensor or None, pointer, bytes)"""
    need = _room(query, name, m, n, k, dt)
    if not need:
        return None, None, 0
    ws = torch.empty(need, dtype=torch.uint8, device=dev)
    return ws, ws.data_ptr(), need


def _matmul(a, b, form, out, dt, ldo):
    (m, k), n = a.codes.shape, b.codes.shape[0]
    dev = out.device
    ws, ptr, size = _workspace(LIB.qopt_fp8_matmul_workspace, "qopt_fp8_matmul_workspace", m, n, k, dt, dev)
    _lib.call("qopt_fp8_matmul", dev, a.codes.data_ptr(), a.scales.data_ptr(), b.codes.data_ptr(),
              b.scales.data_ptr(), form, m, n, k, out.data_ptr(), dt, ldo, ptr, size)
    return out


def _linear(x, dx, m, k, ldx, w, form, out, do, ldo):
    n, dev = w.codes.shape[0], out.device
    ws, ptr, size = None, None, 0
    if m > QOPT_FP8_FEW_ROWS:
        ws, ptr, size = _workspace(LIB.qopt_fp8_linear_workspace, "qopt_fp8_linear_workspace", m, n, k, do, dev)
    _lib.call("qopt_fp8_linear", dev, x.data_ptr(), dx, m, k, ldx, w.codes.data_ptr(),
              w.scales.data_ptr(), form, n, out.data_ptr(), do, ldo, ptr, size)
    return out


# Each of these is one call of the library, without derivatives: torch records nothing of it.  In a
# trace only the empty results would remain, so a trace is refused.

def _not_traced():
    if _is_tracing():
        raise RuntimeError("a library call cannot be traced; the forward passes of fp8_linear, fp4_linear and "
                           "layer_norm can")


def qopt_fp8_quantize(x, *, tiles=False, normal=True, transposed=False):
    """Quantize a 2-D float32 or bfloat16 tensor in blocks of 128 along its rows, or in
    tiles of 128 x 128 (``tiles``).  Returns the Fp8Matrix of x (``normal``), of its transpose
    (``transposed``), or the pair of both."""
    _not_traced()
    if x.dim() != 2:
        raise ValueError("x must be 2-D")
    if not normal and not transposed:
        raise ValueError("nothing to return")
    dt = _check_dtype(x.dtype, "x")
    _same_gpu(x)
    a, b = _quantize(x, dt, _row_stride(x, "x"), tiles, normal, transposed)
    return (a, b) if normal and transposed else a if normal else b


def _span(t):
    """First byte and end of the memory that a tensor's elements lie in."""
    at = t.data_ptr()
    if not t.numel():
        return at, at
    return at, at + (sum((n - 1) * s for n, s in zip(t.shape, t.stride())) + 1) * t.element_size()


def _side_by_side(a, b):
    """Whether two 2-D tensors lie in different columns of rows that are equally far apart."""
    if a.dim() != 2 or b.dim() != 2 or any(t.shape[1] > 1 and t.stride(1) != 1 for t in (a, b)):
        return False
    pitch, of_b = (t.stride(0) * t.element_size() for t in (a, b))
    if pitch != of_b or not pitch:
        return False
    off = (b.data_ptr() - a.data_ptr()) % pitch  # from a row of a to the next one of b
    return a.shape[1] * a.element_size() <= off and off + b.shape[1] * b.element_size() <= pitch


def _output(out, shape, dtype, dev, *operands):
    """The output tensor and the distance of its rows."""
    if out is None:
        return torch.empty(shape, dtype=dtype, device=dev), shape[-1]
    shape = torch.Size(shape)
    if out.shape != shape or out.dtype != dtype:
        raise ValueError(f"out must have shape {tuple(shape)} and dtype {dtype}")
    if out.device != dev:
        raise ValueError("all tensors must be on the same GPU")
    lo, hi = _span(out)
    for t in operands:
        first, end = _span(t)
        if first < hi and lo < end and not _side_by_side(out, t):
            raise ValueError("out must not overlap an operand")
    if out.dim() == 2:
        return out, _row_stride(out, "out")
    if not out.is_contiguous():
        raise ValueError("out must be 2-D with contiguous rows, or contiguous")
    return out, shape[-1]


def qopt_fp8_matmul(a_codes, a_scales, b_codes, b_scales, out_dtype=torch.bfloat16, *, out=None):
    """a b^T of two quantized matrices [m, k] (scales by rows) and [n, k] (by rows or tiles):
    [m, n] in ``out_dtype`` (bfloat16 or float32), into ``out`` if given, which shares no byte
    with an operand."""
    _not_traced()
    fa, fb = _quantized(a_codes, a_scales, "a"), _quantized(b_codes, b_scales, "b")
    dt = _check_dtype(out_dtype, "out_dtype")
    if fa != QOPT_FP8_ROWS:
        raise ValueError("a must have its scales by rows")
    if b_codes.shape[1] != a_codes.shape[1]:
        raise ValueError("a and b must have the same number of columns")
    dev = _same_gpu(a_codes, a_scales, b_codes, b_scales)
    out, ldo = _output(out, (a_codes.shape[0], b_codes.shape[0]), out_dtype, dev,
                       a_codes, a_scales, b_codes, b_scales)
    return _matmul(Fp8Matrix(a_codes, a_scales), Fp8Matrix(b_codes, b_scales), fb, out, dt, ldo)


def qopt_fp8_linear(x, w_codes, w_scales, out_dtype=None, *, out=None):
    """x w^T for x [..., k] in float32 or bfloat16, quantized on the way, and a quantized
    weight [n, k]: [..., n] in ``out_dtype`` (default: x's), without derivatives.  One launch for
    up to QOPT_FP8_FEW_ROWS rows of x.  ``out`` shares no byte with an operand; it may be other
    columns of the buffer that x's rows lie in."""
    _not_traced()
    form = _quantized(w_codes, w_scales, "w")
    dx = _check_dtype(x.dtype, "x")
    out_dtype = x.dtype if out_dtype is None else out_dtype
    do = _check_dtype(out_dtype, "out_dtype")
    if x.dim() < 1:
        raise ValueError("x must have at least one dimension")
    k, n = x.shape[-1], w_codes.shape[0]
    if _blocks(k) * QOPT_FP8_BLOCK != w_codes.shape[1]:
        raise ValueError(f"x has {k} columns, the weight {w_codes.shape[1]} with its padding")
    if x.dim() == 2:
        ldx = _row_stride(x, "x")
    elif x.is_contiguous():
        ldx = k
    else:
        raise ValueError("x must be 2-D with contiguous rows, or contiguous")
    dev = _same_gpu(x, w_codes, w_scales)
    m = x.shape[0] if x.dim() == 2 else x.shape[:-1].numel()
    out, ldo = _output(out, (*x.shape[:-1], n), out_dtype, dev, x, w_codes, w_scales)
    return _linear(x, dx, m, k, ldx, Fp8Matrix(w_codes, w_scales), form, out, do, ldo)


def _check_linear(x, w):
    _check_dtype(x.dtype, "x")
    _check_dtype(w.dtype, "w")
    if w.dim() != 2 or x.dim() < 1 or x.shape[-1] != w.shape[1]:
        raise ValueError("x must be [..., k] and w [n, k]")
    _same_gpu(x, w)


class Fp8LinearFunction(torch.autograd.Function):
    """y = x w^T with both gradients, every product over e4m3 codes: x and the upstream
    gradient in blocks of 128 along the axis of each sum, w in tiles of 128 x 128.

    The quantized matrices of a pass lie in one buffer, addressed by offsets: 10 tensors fewer to
    make (forward and backward of a small layer 137 us of the host's time instead of 178).  Between
    the passes only the transposes that the gradients read are kept."""

    @staticmethod
    def forward(ctx, x, w):
        _check_linear(x, w)
        need_x, need_w = ctx.needs_input_grad
        lead, (n, k) = [int(d) for d in x.shape[:-1]], (int(d) for d in w.shape)  # tensors, in a trace
        m = math.prod(lead)
        x2, w = x.reshape(m, k).contiguous(), w.contiguous()
        dev, dx, kp = x.device, _DT[x.dtype], _blocks(k) * QOPT_FP8_BLOCK
        w_codes, w_all = _sizes(n, k, True)
        wt_codes, wt_all = _sizes(k, n, True) if need_x else (0, 0)
        x_codes, x_all = _sizes(m, k, False) if need_w else (0, 0)
        xt_codes, xt_all = _sizes(k, m, False) if need_w else (0, 0)
        if need_w:
            ws = _room(LIB.qopt_fp8_matmul_workspace, "qopt_fp8_matmul_workspace", m, n, kp, dx)
        else:
            ws = _room(LIB.qopt_fp8_linear_workspace, "qopt_fp8_linear_workspace", m, n, k, dx)
        kept = torch.empty(wt_all + xt_all, dtype=torch.uint8, device=dev)
        temp = torch.empty(w_all + x_all + ws, dtype=torch.uint8, device=dev)
        y = torch.empty(*lead, n, dtype=x.dtype, device=dev)
        wq, wt = temp.data_ptr(), kept.data_ptr()
        xq, xt = wq + w_all, wt + wt_all
        work = xq + x_all if ws else None
        if n and k:
            _lib.call("qopt_fp8_quantize", dev, w.data_ptr(), _DT[w.dtype], n, k, k, QOPT_FP8_TILES,
                      wq, wq + w_codes, *((wt, wt + wt_codes) if need_x else (None, None)))
        if not need_w:
            _lib.call("qopt_fp8_linear", dev, x2.data_ptr(), dx, m, k, k, wq, wq + w_codes,
                      QOPT_FP8_TILES, n, y.data_ptr(), dx, n, work, ws)
        else:
            if m and k:
                _lib.call("qopt_fp8_quantize", dev, x2.data_ptr(), dx, m, k, k, QOPT_FP8_ROWS,
                          xq, xq + x_codes, xt, xt + xt_codes)
            _lib.call("qopt_fp8_matmul", dev, xq, xq + x_codes, wq, wq + w_codes, QOPT_FP8_TILES, m, n,
                      kp, y.data_ptr(), dx, n, work, ws)
        ctx.x_shape, ctx.dtypes = torch.Size((*lead, k)), (x.dtype, w.dtype)
        ctx.save_for_backward(kept)
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        need_x, need_w = ctx.needs_input_grad
        if not need_x and not need_w:
            return None, None
        _not_traced()
        (kept,) = ctx.saved_tensors
        m, n, k = ctx.x_shape[:-1].numel(), dy.shape[-1], ctx.x_shape[-1]
        dy = dy.reshape(m, n).contiguous()
        if dy.dtype not in _DT:
            dy = dy.float()
        dev = dy.device
        wt_codes, wt_all = _sizes(k, n, True) if need_x else (0, 0)
        xt_codes, _ = _sizes(k, m, False) if need_w else (0, 0)
        q_codes, q_all = _sizes(m, n, False) if need_x else (0, 0)
        t_codes, t_all = _sizes(n, m, False) if need_w else (0, 0)
        n_pad, m_pad = _blocks(n) * QOPT_FP8_BLOCK, _blocks(m) * QOPT_FP8_BLOCK
        name, query = "qopt_fp8_matmul_workspace", LIB.qopt_fp8_matmul_workspace
        dx = dw = None
        ws_x = ws_w = 0
        if need_x:
            dx = torch.empty(ctx.x_shape, dtype=ctx.dtypes[0], device=dev)
            ws_x = _room(query, name, m, k, n_pad, _DT[dx.dtype])
        if need_w:
            dw = torch.empty(n, k, dtype=ctx.dtypes[1], device=dev)
            ws_w = _room(query, name, n, k, m_pad, _DT[dw.dtype])
        temp = torch.empty(q_all + t_all + max(ws_x, ws_w), dtype=torch.uint8, device=dev)
        wt, dq = kept.data_ptr(), temp.data_ptr()
        xt, dt, work = wt + wt_all, dq + q_all, dq + q_all + t_all
        if m and n:
            _lib.call("qopt_fp8_quantize", dev, dy.data_ptr(), _DT[dy.dtype], m, n, n, QOPT_FP8_ROWS,
                      *((dq, dq + q_codes) if need_x else (None, None)),
                      *((dt, dt + t_codes) if need_w else (None, None)))
        if need_x:
            _lib.call("qopt_fp8_matmul", dev, dq, dq + q_codes, wt, wt + wt_codes, QOPT_FP8_TILES, m, k, n_pad,
                      dx.data_ptr(), _DT[dx.dtype], k, work if ws_x else None, ws_x)
        if need_w:
            _lib.call("qopt_fp8_matmul", dev, dt, dt + t_codes, xt, xt + xt_codes, QOPT_FP8_ROWS, n, k, m_pad,
                      dw.data_ptr(), _DT[dw.dtype], k, work if ws_w else None, ws_w)
        return dx, dw


def _has_tangent(*tensors):
    # outside of every dual level, which is asked first, there are none (0.6 us of a call)
    return forward_ad._current_level >= 0 and any(forward_ad.unpack_dual(t).tangent is not None for t in tensors)


def fp8_linear(x, w):
    """x w^T with gradients: x [..., k] and w [n, k] in float32 or bfloat16.  The result and
    x's gradient have x's type, w's gradient has w's.  The weight is quantized anew in every
    call; a server quantizes it once and calls ``qopt_fp8_linear``.  A trace (torch.jit.trace)
    holds it as one operation; forward-mode derivatives are refused (NotImplementedError).  A
    forward and backward pass may be captured into a graph as any of torch's: with no other
    result of the same leaves alive whose backward ran, or will run, outside of it."""
    # a trace records the function as one operation, but of the calls below only their empty outputs;
    # of a tangent the function says that it has no derivative, where they would drop it
    if torch.is_grad_enabled() and (x.requires_grad or w.requires_grad) or _is_tracing() \
            or _has_tangent(x, w):
        return Fp8LinearFunction.apply(x, w)
    _check_linear(x, w)
    wq = _quantize(w.detach().contiguous(), _DT[w.dtype], w.shape[1], True, True, False)[0]
    x = x.detach()
    if x.dim() != 2 or x.stride(1) != 1 or x.stride(0) < x.shape[1]:
        x = x.contiguous()
    return qopt_fp8_linear(x, *wq)


class Fp8Linear(torch.nn.Module):
    """Linear layer without bias whose products, forward and backward, run in 8-bit
    floating point (``fp8_linear``).  The weight itself stays in ``dtype`` (float32 or
    bfloat16), Xavier-uniform from ``seed`` as the Stable Embedding's table; without one the seed
    is drawn from torch's generator, so that layers of one shape start apart."""

    def __init__(self, in_features, out_features, *, device=None, dtype=torch.float32, seed=None):
        super().__init__()
        device = torch.device("cuda", torch.cuda.current_device()) if device is None \
            else torch.device(device)
        self.in_features, self.out_features = int(in_features), int(out_features)
        self.seed = int(torch.randint(1 << 62, (), device="cpu")) if seed is None else int(seed)
        self.weight = torch.nn.Parameter(
            torch.empty(self.out_features, self.in_features, dtype=dtype, device=device))
        self.reset_parameters()

    def reset_parameters(self):
        with torch.no_grad():
            qopt_embedding_xavier_init(self.weight, self.seed)

    @torch.no_grad()
    def pack(self):
        """The weight as ``qopt_fp8_linear`` takes it: quantized in tiles, for serving."""
        return qopt_fp8_quantize(self.weight.contiguous(), tiles=True)

    def forward(self, x):
        return fp8_linear(x, self.weight)

    def extra_repr(self):
        return f"{self.in_features}, {self.out_features}, dtype={self.weight.dtype}"
