"""Layer normalisation of activations: wrappers with the C ABI's names
(include/qopt_norm.h), an autograd function and a torch module.

The YaLM-100B training page ("Stabilizations. LayerNorm") puts it in front of a block's
products as well as behind the embedding, where ``StableEmbedding`` has it.  Every step runs
in libqopt's HIP kernels; torch allocates outputs and workspaces and supplies the current
stream.
"""

import ctypes
import math
from functools import lru_cache

import torch
from torch.autograd.function import once_differentiable

from . import _lib
from ._lib import LIB, QOPT_F32
from .fp8 import _DT, _check_dtype, _has_tangent, _is_tracing, _not_traced, _output, _row_stride, _same_gpu


def _check_rows(x, what):
    """(rows, dim, elements between rows) of a tensor [..., dim]."""
    if x.dim() < 1:
        raise ValueError(f"{what} must have at least one dimension")
    if x.dim() == 2:
        return (*x.shape, _row_stride(x, what))
    if not x.is_contiguous():
        raise ValueError(f"{what} must be 2-D with contiguous rows, or contiguous")
    return math.prod(x.shape[:-1]), x.shape[-1], x.shape[-1]


def _check_affine(dim, weight, bias):
    """dtype code of weight and bias (which may be None)."""
    dt = QOPT_F32
    for t, what in ((bias, "bias"), (weight, "weight")):
        if t is not None:
            dt = _check_dtype(t.dtype, what)
            if t.shape != (dim,) or not t.is_contiguous():
                raise ValueError(f"{what} must be contiguous [{dim}]")
    if weight is not None and bias is not None and weight.dtype != bias.dtype:
        raise TypeError("weight and bias must have the same dtype")
    return dt


def _ptr(t):
    return None if t is None else t.data_ptr()


def _eps(eps):
    eps = float(eps)
    if not 0.0 <= eps < math.inf:
        raise ValueError(f"invalid epsilon {eps}")
    return eps


@lru_cache(maxsize=1024)
def _room(rows, dim):
    """Bytes of the backward pass's workspace."""
    need = ctypes.c_size_t(0)
    _lib.check("qopt_layer_norm_backward_workspace",
               LIB.qopt_layer_norm_backward_workspace(rows, dim, ctypes.byref(need)))
    return need.value


# The launches behind the functions below, for operands that are known to be right; mean and rstd as addresses.

def _forward(x, dx, rows, dim, ldx, weight, bias, dw, eps, out, ldo, mean, rstd):
    if rows and dim:
        _lib.call("qopt_layer_norm_forward", x.device, x.data_ptr(), dx, rows, dim, ldx, _ptr(weight),
                  _ptr(bias), dw, eps, out.data_ptr(), ldo, mean, rstd)


def _backward(x, dx, rows, dim, ldx, weight, dw, mean, rstd, dout, lddo, need_x, need_w, need_b, w_dtype):
    dev = x.device
    gx = torch.empty_like(x, memory_format=torch.contiguous_format) if need_x else None
    gw = torch.empty(dim, dtype=w_dtype, device=dev) if need_w else None
    gb = torch.empty(dim, dtype=w_dtype, device=dev) if need_b else None
    ws, size = None, 0
    if need_w or need_b:
        size = _room(rows, dim)
        ws = torch.empty(size, dtype=torch.uint8, device=dev)
    if dim:
        _lib.call("qopt_layer_norm_backward", dev, x.data_ptr(), dx, rows, dim, ldx, _ptr(weight), dw,
                  mean, rstd, dout.data_ptr(), lddo, _ptr(gx), dim, _ptr(gw), _ptr(gb),
                  ws.data_ptr() if size else None, size)
    return gx, gw, gb


# Each of these is one call of the library, without derivatives: torch records nothing of it.

def qopt_layer_norm_forward(x, weight=None, bias=None, eps=1e-5, *, save_stats=True, out=None):
    """The rows of x [..., dim] (float32 or bfloat16) normalised, times ``weight`` plus ``bias``
    ([dim], both float32 or both bfloat16).  Returns (out, mean, rstd), out in x's shape and type, the
    others float32, one value per row (None unless ``save_stats``; NaN for rows without values).  ``out`` may be passed in;
    it shares no byte with an operand, but may be other columns of the buffer that x lies in."""
    _not_traced()
    dx = _check_dtype(x.dtype, "x")
    rows, dim, ldx = _check_rows(x, "x")
    dw = _check_affine(dim, weight, bias)
    eps = _eps(eps)
    operands = [t for t in (x, weight, bias) if t is not None]
    dev = _same_gpu(*operands)
    out, ldo = _output(out, tuple(x.shape), x.dtype, dev, *operands)
    mean = rstd = None
    if save_stats:
        mean, rstd = torch.empty(2, rows, dtype=torch.float32, device=dev) if dim else \
            torch.full((2, rows), math.nan, dtype=torch.float32, device=dev)
    _forward(x, dx, rows, dim, ldx, weight, bias, dw, eps, out, ldo, _ptr(mean), _ptr(rstd))
    return out, mean, rstd


def qopt_layer_norm_backward(x, weight, mean, rstd, dout, *, need_x=True, need_weight=True, need_bias=True,
                             weight_dtype=None):
    """Gradients for the upstream ``dout`` (x's shape and type) from x and the statistics that
    ``qopt_layer_norm_forward`` returned: (dx, dweight, dbias), each None where it is not needed.  The last
    two have ``weight_dtype`` (default: the weight's, float32 without one)."""
    _not_traced()
    dx = _check_dtype(x.dtype, "x")
    rows, dim, ldx = _check_rows(x, "x")
    _check_affine(dim, weight, None)
    if weight_dtype is None:
        weight_dtype = torch.float32 if weight is None else weight.dtype
    dw = _check_dtype(weight_dtype, "weight_dtype")
    if weight is not None and weight.dtype != weight_dtype:
        raise TypeError("weight_dtype must be the weight's")
    if dout.shape != x.shape or dout.dtype != x.dtype:
        raise ValueError("dout must have x's shape and dtype")
    for t in (mean, rstd):
        if t.dtype != torch.float32 or t.numel() != rows or not t.is_contiguous():
            raise ValueError("mean and rstd must be contiguous float32, one value per row")
    _same_gpu(*(t for t in (x, weight, mean, rstd, dout) if t is not None))
    lddo = _check_rows(dout, "dout")[2]
    return _backward(x, dx, rows, dim, ldx, weight, dw, mean.data_ptr(), rstd.data_ptr(), dout, lddo, need_x,
                     need_weight, need_bias, weight_dtype)


def _check_layer(x, weight, bias):
    _check_dtype(x.dtype, "x")
    if x.dim() < 1:
        raise ValueError("x must have at least one dimension")
    wanted = x.shape[-1:]
    for t, what in ((bias, "bias"), (weight, "weight")):
        if t is not None:
            _check_dtype(t.dtype, what)
            if t.shape != wanted:
                raise ValueError(f"{what} must be [{wanted[0]}]")
    if weight is not None and bias is not None and weight.dtype != bias.dtype:
        raise TypeError("weight and bias must have the same dtype")
    _same_gpu(*(t for t in (x, weight, bias) if t is not None))


class LayerNormFunction(torch.autograd.Function):
    """Layer normalisation over the last axis with gradients for x, the weight and the bias."""

    @staticmethod
    def forward(ctx, x, weight, bias, eps):
        _check_layer(x, weight, bias)
        eps = _eps(eps)
        x, weight, bias = (t if t is None or t.is_contiguous() else t.contiguous() for t in (x, weight, bias))
        dim = int(x.shape[-1])
        rows = math.prod(int(d) for d in x.shape[:-1])  # tensors, in a trace
        some = weight if weight is not None else bias
        dw = QOPT_F32 if some is None else _DT[some.dtype]
        y = torch.empty_like(x)
        stats = torch.empty(2, rows, dtype=torch.float32, device=x.device)
        _forward(x, _DT[x.dtype], rows, dim, dim, weight, bias, dw, eps, y, dim,
                 stats.data_ptr(), stats.data_ptr() + 4 * rows)
        ctx.w_dtype = torch.float32 if some is None else some.dtype
        ctx.rows = rows
        ctx.save_for_backward(x, weight, stats)
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dout):
        need = ctx.needs_input_grad
        if not any(need):
            return None, None, None, None
        _not_traced()
        x, weight, stats = ctx.saved_tensors
        dim = x.shape[-1]
        dout = dout.contiguous()
        if dout.dtype != x.dtype:
            dout = dout.to(x.dtype)
        gx, gw, gb = _backward(x, _DT[x.dtype], ctx.rows, dim, dim, weight, _DT[ctx.w_dtype], stats.data_ptr(),
                               stats.data_ptr() + 4 * ctx.rows, dout, dim, need[0], need[1], need[2], ctx.w_dtype)
        return gx, gw, gb, None


def layer_norm(x, weight=None, bias=None, eps=1e-5):
    """Layer normalisation over the last axis of x (float32 or bfloat16), times ``weight`` plus
    ``bias`` ([dim], both float32 or both bfloat16; either may be None), with gradients for all three.  A
    trace (torch.jit.trace) holds it as one operation; forward-mode derivatives are refused
    (NotImplementedError).  For passes that are captured into a graph the conditions of
    ``fp8_linear`` hold."""
    given = [t for t in (x, weight, bias) if t is not None]
    if torch.is_grad_enabled() and any(t.requires_grad for t in given) or _is_tracing() or _has_tangent(*given):
        return LayerNormFunction.apply(x, weight, bias, eps)
    _check_layer(x, weight, bias)
    given = [None if t is None else t.detach() for t in (x, weight, bias)]
    x, weight, bias = (t if t is None or t.is_contiguous() else t.contiguous() for t in given)
    return qopt_layer_norm_forward(x, weight, bias, eps, save_stats=False)[0]


class LayerNorm(torch.nn.Module):
    """Layer normalisation over a last axis of ``dim`` values (``layer_norm``), weight 1 and bias 0 at
    first, both in ``dtype`` (float32 or bfloat16); ``bias=False`` leaves the bias out."""

    def __init__(self, dim, eps=1e-5, *, bias=True, device=None, dtype=torch.float32):
        super().__init__()
        device = torch.device("cuda", torch.cuda.current_device()) if device is None \
            else torch.device(device)
        _check_dtype(dtype, "dtype")
        self.dim, self.eps = int(dim), _eps(eps)
        self.weight = torch.nn.Parameter(torch.empty(self.dim, dtype=dtype, device=device))
        if bias:
            self.bias = torch.nn.Parameter(torch.empty(self.dim, dtype=dtype, device=device))
        else:
            self.register_parameter("bias", None)
        self.reset_parameters()

    def reset_parameters(self):
        with torch.no_grad():
            self.weight.fill_(1.0)
            if self.bias is not None:
                self.bias.zero_()

    def forward(self, x):
        return layer_norm(x, self.weight, self.bias, self.eps)

    def extra_repr(self):
        return f"{self.dim}, eps={self.eps}, bias={self.bias is not None}, dtype={self.weight.dtype}"
