"""Linear products in microscaled 4-bit floating point: wrappers with the C ABI's names
(include/qopt_fp4.h), an autograd function and a torch module.

e2m1 codes with one power-of-two scale per 32 values along the summed axis, for activations
and weights alike: a weight of 17 bits per 32 where ``fp8`` keeps 8 bits per value.
``fp4_linear`` trains a weight that will be served in 4 bits: its forward pass is the product
that a server computes, its gradients are straight-through (the quantization counts as the
identity) and run in the 8-bit products of include/qopt_fp8.h, whose blocks hold what an
upstream gradient spreads over.  Every step runs in libqopt's HIP kernels; torch allocates
outputs and workspaces and supplies the current stream.
"""

import math
from typing import NamedTuple

import torch
from torch.autograd.function import once_differentiable

from . import _lib
from ._lib import LIB, QOPT_FP4_FEW_ROWS, QOPT_FP4_PAD, QOPT_FP8_ROWS, QOPT_FP8_TILES
from .embedding import qopt_embedding_xavier_init
from .fp8 import (_DT, _check_dtype, _check_linear, _has_tangent, _is_tracing, _not_traced, _output, _room,
                  _row_stride, _same_gpu, _sizes as _sizes8, _workspace)


class Fp4Matrix(NamedTuple):
    """A quantized matrix: uint8 codes [rows, K / 2], K the columns up to a multiple of 256 and
    the even column's code in the low half of a byte, and uint8 scales [K / 128, rows up to a
    multiple of 16, 4], each standing for 2^(scale - 127) and 32 values of a row."""
    codes: torch.Tensor
    scales: torch.Tensor


def _padded(cols):
    return -(-int(cols) // QOPT_FP4_PAD) * QOPT_FP4_PAD


def _padded_rows(rows):
    return -(-int(rows) // 16) * 16


def _quantized(codes, scales, what):
    """Checks a (codes, scales) pair; returns (rows, padded columns)."""
    if codes.dtype is not torch.uint8 or scales.dtype is not torch.uint8:
        raise TypeError(f"{what}: codes and scales must be uint8")
    if codes.dim() != 2 or 2 * codes.shape[1] % QOPT_FP4_PAD:
        raise ValueError(f"{what}: codes must be 2-D with a multiple of {QOPT_FP4_PAD // 2} columns")
    rows, k = codes.shape[0], 2 * codes.shape[1]
    if not codes.is_contiguous() or not scales.is_contiguous():
        raise ValueError(f"{what}: codes and scales must be contiguous")
    if scales.shape != (k // 128, _padded_rows(rows), 4):
        raise ValueError(f"{what}: scales must be {(k // 128, _padded_rows(rows), 4)}, not {tuple(scales.shape)}")
    return rows, k


# The launches behind the functions below, for operands that are known to be right.

def _quantize(x, dt, ldx):
    rows, cols = x.shape
    k = _padded(cols)
    codes = torch.empty(rows, k // 2, dtype=torch.uint8, device=x.device)
    scales = torch.empty(k // 128, _padded_rows(rows), 4, dtype=torch.uint8, device=x.device)
    if rows and cols:
        _lib.call("qopt_fp4_quantize", x.device, x.data_ptr(), dt, rows, cols, ldx, codes.data_ptr(), scales.data_ptr())
    return Fp4Matrix(codes, scales)


def _sizes(rows, cols):
    """Bytes of the codes of a quantized matrix, and of both its parts up to a whole page."""
    k = _padded(cols)
    codes = rows * k // 2
    return codes, -(-(codes + k // 128 * _padded_rows(rows) * 4) // 4096) * 4096


def _linear(x, dx, m, k, ldx, w, out, do, ldo):
    n, dev = w.codes.shape[0], out.device
    ws, ptr, size = None, None, 0
    if m > QOPT_FP4_FEW_ROWS:
        ws, ptr, size = _workspace(LIB.qopt_fp4_linear_workspace, "qopt_fp4_linear_workspace", m, n, k, do, dev)
    _lib.call("qopt_fp4_linear", dev, x.data_ptr(), dx, m, k, ldx, w.codes.data_ptr(), w.scales.data_ptr(), n,
              out.data_ptr(), do, ldo, ptr, size)
    return out


# Each of these is one call of the library, without derivatives: torch records nothing of it.

def qopt_fp4_quantize(x):
    """Quantize a 2-D float32 or bfloat16 tensor in blocks of 32 along its rows: an Fp4Matrix."""
    _not_traced()
    if x.dim() != 2:
        raise ValueError("x must be 2-D")
    dt = _check_dtype(x.dtype, "x")
    _same_gpu(x)
    return _quantize(x, dt, _row_stride(x, "x"))


def qopt_fp4_dequantize(codes, scales, columns, dtype=torch.float32, *, out=None):
    """The values [rows, columns] that a quantized matrix stands for, in ``dtype`` (float32 or
    bfloat16), into ``out`` if given, which shares no byte with an operand."""
    _not_traced()
    rows, k = _quantized(codes, scales, "the matrix")
    dt = _check_dtype(dtype, "dtype")
    columns = int(columns)
    if _padded(columns) != k:
        raise ValueError(f"{columns} columns with their padding are not the {k} of the codes")
    dev = _same_gpu(codes, scales)
    out, ldo = _output(out, (rows, columns), dtype, dev, codes, scales)
    if rows and columns:
        _lib.call("qopt_fp4_dequantize", dev, codes.data_ptr(), scales.data_ptr(), rows, columns, out.data_ptr(), dt, ldo)
    return out


def qopt_fp4_matmul(a_codes, a_scales, b_codes, b_scales, out_dtype=torch.bfloat16, *, out=None):
    """a b^T of two quantized matrices [m, k] and [n, k]: [m, n] in ``out_dtype`` (bfloat16 or
    float32), into ``out`` if given, which shares no byte with an operand."""
    _not_traced()
    (m, k), (n, kb) = _quantized(a_codes, a_scales, "a"), _quantized(b_codes, b_scales, "b")
    dt = _check_dtype(out_dtype, "out_dtype")
    if k != kb:
        raise ValueError("a and b must have the same number of columns")
    dev = _same_gpu(a_codes, a_scales, b_codes, b_scales)
    out, ldo = _output(out, (m, n), out_dtype, dev, a_codes, a_scales, b_codes, b_scales)
    ws, ptr, size = _workspace(LIB.qopt_fp4_matmul_workspace, "qopt_fp4_matmul_workspace", m, n, k, dt, dev)
    _lib.call("qopt_fp4_matmul", dev, a_codes.data_ptr(), a_scales.data_ptr(), b_codes.data_ptr(), b_scales.data_ptr(),
              m, n, k, out.data_ptr(), dt, ldo, ptr, size)
    return out


def qopt_fp4_linear(x, w_codes, w_scales, out_dtype=None, *, out=None):
    """x w^T for x [..., k] in float32 or bfloat16, quantized on the way, and a quantized
    weight [n, k]: [..., n] in ``out_dtype`` (default: x's), without derivatives.  One launch for
    up to QOPT_FP4_FEW_ROWS rows of x.  ``out`` shares no byte with an operand; it may be other
    columns of the buffer that x's rows lie in."""
    _not_traced()
    n, kp = _quantized(w_codes, w_scales, "w")
    dx = _check_dtype(x.dtype, "x")
    out_dtype = x.dtype if out_dtype is None else out_dtype
    do = _check_dtype(out_dtype, "out_dtype")
    if x.dim() < 1:
        raise ValueError("x must have at least one dimension")
    k = x.shape[-1]
    if _padded(k) != kp:
        raise ValueError(f"x has {k} columns, the weight {kp} with its padding")
    if x.dim() == 2:
        ldx = _row_stride(x, "x")
    elif x.is_contiguous():
        ldx = k
    else:
        raise ValueError("x must be 2-D with contiguous rows, or contiguous")
    dev = _same_gpu(x, w_codes, w_scales)
    m = x.shape[0] if x.dim() == 2 else x.shape[:-1].numel()
    out, ldo = _output(out, (*x.shape[:-1], n), out_dtype, dev, x, w_codes, w_scales)
    return _linear(x, dx, m, k, ldx, Fp4Matrix(w_codes, w_scales), out, do, ldo)


class Fp4LinearFunction(torch.autograd.Function):
    """y = x w^T over 4-bit codes of both; dx = dy w and dw = dy^T x over 8-bit codes of what was
    given (x and dy in blocks of 128 along the axis of each sum, w in tiles of 128 x 128), as the
    gradients of ``fp8_linear``.  x and w themselves are kept between the passes."""

    @staticmethod
    def forward(ctx, x, w):
        _check_linear(x, w)
        lead, (n, k) = [int(d) for d in x.shape[:-1]], (int(d) for d in w.shape)  # tensors, in a trace
        m = math.prod(lead)
        x2, w = x.reshape(m, k).contiguous(), w.contiguous()
        dev, dx = x.device, _DT[x.dtype]
        w_codes, w_all = _sizes(n, k)
        ws = _room(LIB.qopt_fp4_linear_workspace, "qopt_fp4_linear_workspace", m, n, k, dx)
        temp = torch.empty(w_all + ws, dtype=torch.uint8, device=dev)
        y = torch.empty(*lead, n, dtype=x.dtype, device=dev)
        wq = temp.data_ptr()
        if n and k:
            _lib.call("qopt_fp4_quantize", dev, w.data_ptr(), _DT[w.dtype], n, k, k, wq, wq + w_codes)
        _lib.call("qopt_fp4_linear", dev, x2.data_ptr(), dx, m, k, k, wq, wq + w_codes, n, y.data_ptr(), dx, n,
                  wq + w_all if ws else None, ws)
        need_x, need_w = ctx.needs_input_grad
        ctx.x_shape, ctx.dtypes = torch.Size((*lead, k)), (x.dtype, w.dtype)
        ctx.save_for_backward(x2 if need_w else None, w if need_x else None)
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        need_x, need_w = ctx.needs_input_grad
        if not need_x and not need_w:
            return None, None
        _not_traced()
        x, w = ctx.saved_tensors
        m, n, k = ctx.x_shape[:-1].numel(), dy.shape[-1], ctx.x_shape[-1]
        dy = dy.reshape(m, n).contiguous()
        if dy.dtype not in _DT:
            dy = dy.float()
        dev = dy.device
        n_pad, m_pad = (-(-d // 128) * 128 for d in (n, m))
        name, query = "qopt_fp8_matmul_workspace", LIB.qopt_fp8_matmul_workspace
        # the quantized matrices in one buffer: w^T and dy for dx, dy^T and x^T for dw
        wt_codes, wt_all = _sizes8(k, n, True) if need_x else (0, 0)
        q_codes, q_all = _sizes8(m, n, False) if need_x else (0, 0)
        t_codes, t_all = _sizes8(n, m, False) if need_w else (0, 0)
        xt_codes, xt_all = _sizes8(k, m, False) if need_w else (0, 0)
        dx = dw = None
        ws_x = ws_w = 0
        if need_x:
            dx = torch.empty(ctx.x_shape, dtype=ctx.dtypes[0], device=dev)
            ws_x = _room(query, name, m, k, n_pad, _DT[dx.dtype])
        if need_w:
            dw = torch.empty(n, k, dtype=ctx.dtypes[1], device=dev)
            ws_w = _room(query, name, n, k, m_pad, _DT[dw.dtype])
        temp = torch.empty(wt_all + q_all + t_all + xt_all + max(ws_x, ws_w), dtype=torch.uint8, device=dev)
        wt = temp.data_ptr()
        dq = wt + wt_all
        dt = dq + q_all
        xt = dt + t_all
        work = xt + xt_all
        if m and n:
            _lib.call("qopt_fp8_quantize", dev, dy.data_ptr(), _DT[dy.dtype], m, n, n, QOPT_FP8_ROWS,
                      *((dq, dq + q_codes) if need_x else (None, None)),
                      *((dt, dt + t_codes) if need_w else (None, None)))
        if need_x:
            if n and k:
                _lib.call("qopt_fp8_quantize", dev, w.data_ptr(), _DT[w.dtype], n, k, k, QOPT_FP8_TILES,
                          None, None, wt, wt + wt_codes)
            _lib.call("qopt_fp8_matmul", dev, dq, dq + q_codes, wt, wt + wt_codes, QOPT_FP8_TILES, m, k, n_pad,
                      dx.data_ptr(), _DT[dx.dtype], k, work if ws_x else None, ws_x)
        if need_w:
            if m and k:
                _lib.call("qopt_fp8_quantize", dev, x.data_ptr(), _DT[x.dtype], m, k, k, QOPT_FP8_ROWS,
                          None, None, xt, xt + xt_codes)
            _lib.call("qopt_fp8_matmul", dev, dt, dt + t_codes, xt, xt + xt_codes, QOPT_FP8_ROWS, n, k, m_pad,
                      dw.data_ptr(), _DT[dw.dtype], k, work if ws_w else None, ws_w)
        return dx, dw


def fp4_linear(x, w):
    """x w^T over 4-bit codes, with straight-through gradients: x [..., k] and w [n, k] in
    float32 or bfloat16.  The result and x's gradient have x's type, w's gradient has w's; the
    gradients are ``fp8_linear``'s, with what its 8-bit products lose in bfloat16 ones (qopt_fp8.h).  The
    weight is quantized anew in every call; a server quantizes it once and calls
    ``qopt_fp4_linear``, which gives the same result.  A trace (torch.jit.trace) holds it as one
    operation; forward-mode derivatives are refused (NotImplementedError).  For passes that are
    captured into a graph the conditions of ``fp8_linear`` hold."""
    if torch.is_grad_enabled() and (x.requires_grad or w.requires_grad) or _is_tracing() \
            or _has_tangent(x, w):
        return Fp4LinearFunction.apply(x, w)
    _check_linear(x, w)
    w = w.detach().contiguous()
    wq = _quantize(w, _DT[w.dtype], w.shape[1])
    x = x.detach()
    if x.dim() != 2 or x.stride(1) != 1 or x.stride(0) < x.shape[1]:
        x = x.contiguous()
    return qopt_fp4_linear(x, *wq)


class Fp4Linear(torch.nn.Module):
    """Linear layer without bias whose product runs in microscaled 4-bit floating point
    (``fp4_linear``).  The weight itself stays in ``dtype`` (float32 or bfloat16), Xavier-uniform
    from ``seed`` as the Stable Embedding's table; without one the seed is drawn from torch's
    generator, so that layers of one shape start apart."""

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
        """The weight as ``qopt_fp4_linear`` takes it, for serving."""
        return qopt_fp4_quantize(self.weight.contiguous())

    def forward(self, x):
        return fp4_linear(x, self.weight)

    def extra_repr(self):
        return f"{self.in_features}, {self.out_features}, dtype={self.weight.dtype}"
