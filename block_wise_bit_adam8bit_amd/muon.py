"""Muon: steps of a model's matrices along their orthogonalised momentum, with the momentum
held as block-wise dynamic-tree 8-bit codes or in fp32.

Wrappers with the C ABI's names (include/qopt_muon.h) and a torch optimizer that stands next
to ``AdamW``: matrices here, vectors and embeddings there.  The 8-bit state is the first moment
of the 8-bit optimizers summary page (signed codebook, blocks of 2048 with their own absmax).
Every step runs in libqopt's HIP kernels; torch allocates state and workspaces and supplies
the current stream.
"""

import ctypes
import math
from collections import defaultdict

import torch

from . import _lib
from ._lib import LIB, QOPT_F32, QOPT_MUON_MATCH_RMS_ADAMW, QOPT_MUON_MAX_DIM, QOPT_MUON_MAX_STEPS, QOPT_MUON_ORIGINAL
from .fp8 import _check_dtype, _not_traced, _output, _same_gpu
from .functional import (SIGNED, _check_grad_scale, _check_spans, codebook, nblocks, qopt_dequantize_blockwise,
                         qopt_quantize_blockwise)
from .optim import _CODE_ALIGN, _MOMENT_ALIGN, Adam8bit

_DT = {torch.float32: _lib.QOPT_F32, torch.bfloat16: _lib.QOPT_BF16}
_ADJUST = {"original": QOPT_MUON_ORIGINAL, "match_rms_adamw": QOPT_MUON_MATCH_RMS_ADAMW}


def _check_iterations(steps, eps):
    if int(steps) != steps or not 1 <= steps <= QOPT_MUON_MAX_STEPS:
        raise ValueError(f"steps must be 1 to {QOPT_MUON_MAX_STEPS}, not {steps}")
    if not 0.0 < eps < math.inf:
        raise ValueError(f"invalid epsilon {eps}")


def qopt_orthogonalize(x, *, steps=5, eps=1e-7, out_dtype=None, out=None):
    """Newton-Schulz iterations on the matrices x [..., rows, cols] (float32 or bfloat16,
    contiguous), each divided by the larger of its Frobenius norm and ``eps``: x's shape in
    ``out_dtype`` (default: x's), without derivatives, into ``out`` if given, which shares no
    byte with x."""
    _not_traced()
    dx = _check_dtype(x.dtype, "x")
    out_dtype = x.dtype if out_dtype is None else out_dtype
    do = _check_dtype(out_dtype, "out_dtype")
    if x.dim() < 2:
        raise ValueError("x must be [..., rows, cols]")
    if not x.is_contiguous():
        raise ValueError("x must be contiguous")
    _check_iterations(steps, eps)
    dev = _same_gpu(x)
    *lead, rows, cols = x.shape
    batch = math.prod(lead)
    if max(rows, cols) > QOPT_MUON_MAX_DIM:
        raise ValueError(f"matrices of at most {QOPT_MUON_MAX_DIM} rows or columns")
    if out is not None and not out.is_contiguous():
        raise ValueError("out must be contiguous")
    out, _ = _output(out, tuple(x.shape), out_dtype, dev, x)
    if x.numel():
        need = ctypes.c_size_t(0)
        _lib.check("qopt_orthogonalize_workspace",
                   LIB.qopt_orthogonalize_workspace(batch, rows, cols, ctypes.byref(need)))
        ws = torch.empty(need.value, dtype=torch.uint8, device=dev)
        _lib.call("qopt_orthogonalize", dev, x.data_ptr(), dx, batch, rows, cols, int(steps), float(eps),
                  out.data_ptr(), do, ws.data_ptr(), need.value)
    return out


class MuonPlan:
    """The checked tensors of a Muon step over one list of matrices, made by
    qopt_muon8bit_plan or qopt_muon32bit_plan and stepped any number of times.  It keeps the
    memory that the tensors had when it was made and steps that memory: a tensor that is given
    other memory later (``p.data = ...``) needs a new plan."""

    __slots__ = ("bits", "tensors", "storages", "array", "pdtype", "gdtype", "device", "room")

    def __init__(self, bits, tensors, array, pdtype, gdtype, device, room):
        self.bits, self.tensors, self.array = bits, tensors, array
        self.pdtype, self.gdtype, self.device, self.room = pdtype, gdtype, device, room
        self.storages = ()

    def keep(self):
        """Hold the tensors' memory too, for a plan that is stepped more than once."""
        self.storages = [x.untyped_storage() for t in self.tensors for x in t]
        return self


def _muon_plan(tensors, bits):
    """Checks the tuples of a Muon step and makes its descriptors."""
    tensors = [tuple(t) for t in tensors]
    coded = bits == 8
    arr = (_lib.qopt_muon_tensor * len(tensors))()
    pair = device = None
    spans = []
    for i, t in enumerate(tensors):
        if len(t) != (4 if coded else 3):
            raise ValueError("each item must be (param, grad, m_codes, m_absmax)" if coded
                             else "each item must be (param, grad, m)")
        p, g, m = t[:3]
        if p.dim() != 2 or g.shape != p.shape:
            raise ValueError("params must be matrices, with gradients of their shape")
        if max(p.shape) > QOPT_MUON_MAX_DIM:
            raise ValueError(f"matrices of at most {QOPT_MUON_MAX_DIM} rows or columns")
        if p.dtype not in _DT or g.dtype not in _DT:
            raise TypeError("params and grads must be float32 or bfloat16")
        if pair is None:
            pair = p.dtype, g.dtype
        elif (p.dtype, g.dtype) != pair:
            raise TypeError("one call takes one (param dtype, grad dtype) pair")
        n = p.numel()
        if m.numel() != n:
            raise ValueError("param and momentum must have the same size")
        if coded:
            if m.dtype != torch.uint8 or t[3].dtype != torch.float32:
                raise TypeError("codes must be uint8 and absmax float32")
            if t[3].numel() != nblocks(n):
                raise ValueError("absmax must hold ceil(n / 2048) elements")
        elif m.dtype != torch.float32:
            raise TypeError("momentum must be float32")
        d = _same_gpu(*t)
        if device is None:
            device = d
        elif d != device:
            raise ValueError("all tensors of one call must be on the same GPU")
        for x in t:
            if not x.is_contiguous():
                raise ValueError("tensors must be contiguous")
        arr[i] = (p.data_ptr(), g.data_ptr(), m.data_ptr(), t[3].data_ptr() if coded else None, *p.shape)
        if n:
            spans += ((x.data_ptr(), x.data_ptr() + x.numel() * x.element_size(), j != 1)  # all but the gradient
                      for j, x in enumerate(t))
    _check_spans(spans)
    need = ctypes.c_size_t(0)
    _lib.check("qopt_muon_workspace", LIB.qopt_muon_workspace(arr, len(arr), ctypes.byref(need)))
    pdt, gdt = (QOPT_F32, QOPT_F32) if pair is None else (_DT[pair[0]], _DT[pair[1]])
    return MuonPlan(bits, tensors, arr, pdt, gdt, device, need.value)


def qopt_muon8bit_plan(tensors):
    """Plan of a Muon step with 8-bit momentum over a list of (param, grad, m_codes, m_absmax)
    tuples: matrices of any shapes, fp32 or bf16 params and grads; none may overlap another."""
    plan = _muon_plan(tensors, 8)
    if plan.device is not None:
        codebook(SIGNED, plan.device)  # a step may be captured from here on
    return plan.keep()


def qopt_muon32bit_plan(tensors):
    """Plan of a Muon step with fp32 momentum over a list of (param, grad, m) tuples; none may
    overlap another."""
    return _muon_plan(tensors, 32).keep()


def _settings(lr, momentum, weight_decay, nesterov, adjust, steps, eps):
    if adjust not in _ADJUST:
        raise ValueError(f"adjust must be one of {sorted(_ADJUST)}, not {adjust!r}")
    _check_iterations(steps, eps)
    return _lib.qopt_muon_hparams(float(lr), float(momentum), float(weight_decay), float(eps), 1 if nesterov else 0,
                                  _ADJUST[adjust], int(steps))


def _check_settings(**settings):
    """Refuse hyper-parameters as the library does: it checks them also for a step of no tensors."""
    _lib.check("qopt_muon32bit_step", LIB.qopt_muon32bit_step(
        None, 0, QOPT_F32, QOPT_F32, ctypes.byref(_settings(**settings)), None, None, 0, None))


def _muon_step(tensors, bits, grad_scale, settings):
    plan = tensors if isinstance(tensors, MuonPlan) else _muon_plan(tensors, bits)
    if plan.bits != bits:
        raise ValueError(f"the plan is one of a step with {plan.bits}-bit momentum")
    _not_traced()
    _check_grad_scale(grad_scale)
    dev = plan.device
    if grad_scale is not None and dev is not None and grad_scale.device != dev:
        raise ValueError("grad_scale must be on the tensors' GPU")
    hp = _settings(**settings)
    if dev is None:
        _check_settings(**settings)
        return
    ws = torch.empty(plan.room, dtype=torch.uint8, device=dev)
    _lib.call(f"qopt_muon{bits}bit_step", dev, plan.array, len(plan.array), plan.pdtype, plan.gdtype,
              *((codebook(SIGNED, dev).data_ptr(),) if bits == 8 else ()), ctypes.byref(hp),
              None if grad_scale is None else grad_scale.data_ptr(), ws.data_ptr() if plan.room else None, plan.room)


def qopt_muon8bit_step(tensors, *, lr, momentum, weight_decay, nesterov=True, adjust="original", steps=5, eps=1e-7,
                       grad_scale=None):
    """One Muon step with 8-bit momentum over a list of (param, grad, m_codes, m_absmax) tuples,
    or a plan of it, updated in place on torch's current stream.  ``adjust``: "original" (rate lr
    sqrt(max(1, rows / cols))) or "match_rms_adamw" (lr 0.2 sqrt(max(rows, cols))); ``steps``,
    ``eps``: those of qopt_orthogonalize; ``grad_scale``: a float32 GPU tensor of one value that
    every gradient is multiplied with, read when the step runs."""
    _muon_step(tensors, 8, grad_scale, dict(lr=lr, momentum=momentum, weight_decay=weight_decay, nesterov=nesterov,
                                            adjust=adjust, steps=steps, eps=eps))


def qopt_muon32bit_step(tensors, *, lr, momentum, weight_decay, nesterov=True, adjust="original", steps=5, eps=1e-7,
                        grad_scale=None):
    """One Muon step with fp32 momentum over a list of (param, grad, m) tuples, or a plan of it,
    updated in place on torch's current stream; the settings as for qopt_muon8bit_step."""
    _muon_step(tensors, 32, grad_scale, dict(lr=lr, momentum=momentum, weight_decay=weight_decay, nesterov=nesterov,
                                             adjust=adjust, steps=steps, eps=eps))


_CODED_KEYS = ("m_codes", "m_absmax")
_BUFFER_KEYS = ("momentum_buffer",)


def _flat_state(device, shapes, coded):
    """Zero-filled momentum per parameter shape, views of one flat buffer per kind."""
    align, off, blk, c, b = (_CODE_ALIGN if coded else _MOMENT_ALIGN), [], [], 0, 0
    for s in shapes:
        off.append(c)
        blk.append(b)
        c += -(-s.numel() // align) * align
        b += nblocks(s.numel())
    m = torch.zeros(max(c, 1), dtype=torch.uint8 if coded else torch.float32, device=device)
    views = [m[o:o + s.numel()].view(s) for s, o in zip(shapes, off)]
    if not coded:
        return [(v,) for v in views]
    if device.type == "cuda":
        codebook(SIGNED, device)  # a step may be captured from here on
    am = torch.zeros(max(b, 1), dtype=torch.float32, device=device)
    return [(v.view(-1), am[k:k + nblocks(v.numel())]) for v, k in zip(views, blk)]


class Muon(torch.optim.Optimizer):
    """Muon for a model's matrices (2-D parameters), momentum held in 8 bits or in 32.

    ``state_bits`` (8 or 32) and ``min_8bit_size`` are per-group options as in ``AdamW``.  The
    update is that of ``torch.optim.Muon`` (exponential average, Nesterov, Newton-Schulz with
    its coefficients, decoupled weight decay, ``adjust`` as its ``adjust_lr_fn``), with the
    orthogonalisation at the precision of qopt_orthogonalize.  Parameters and gradients must be
    contiguous float32 or bfloat16 GPU tensors; all matrices of a group, device and type take one
    fused step.  ``step(grad_scale=t)`` multiplies every gradient with the float32 GPU value
    ``t`` inside the step.  A step that begins states is not captured into a graph; a captured one
    keeps its settings and the memory of its parameters, gradients and state: loading a state dict gives
    the state other memory, behind which a step is captured anew.

    A step takes a workspace from torch's allocator and gives it back at its end: 12 bytes per element of
    the matrices that share their launches (at most 16 of more than 128 rows and columns, or until their
    products fill the chip), 20 per value of their m x m, m the shorter side, and up to 0.14 GB of partial
    sums, so 1.0 GB for one matrix of 4096 x 11008, however many bits its momentum has.
    """

    def __init__(self, params, lr=1e-3, momentum=0.95, weight_decay=0.1, *, nesterov=True, adjust="original",
                 ns_steps=5, eps=1e-7, state_bits=8, min_8bit_size=4096):
        super().__init__(params, dict(lr=lr, momentum=momentum, weight_decay=weight_decay, nesterov=nesterov,
                                      adjust=adjust, ns_steps=ns_steps, eps=eps, state_bits=state_bits,
                                      min_8bit_size=min_8bit_size))

    @staticmethod
    def _group_settings(g):
        return dict(lr=float(g["lr"]), momentum=g["momentum"], weight_decay=g["weight_decay"],
                    nesterov=g["nesterov"], adjust=g["adjust"], steps=g["ns_steps"], eps=g["eps"])

    def add_param_group(self, param_group):
        g = {**self.defaults, **param_group}
        if not 0.0 <= g["lr"]:
            raise ValueError(f"invalid learning rate {g['lr']}")
        if not 0.0 <= g["momentum"] < 1.0:
            raise ValueError(f"invalid momentum {g['momentum']}")
        if not 0.0 <= g["weight_decay"]:
            raise ValueError(f"invalid weight decay {g['weight_decay']}")
        if g["state_bits"] not in (8, 32):
            raise ValueError(f"state_bits must be 8 or 32, not {g['state_bits']}")
        _settings(**self._group_settings(g))
        super().add_param_group(param_group)
        for p in self.param_groups[-1]["params"]:
            if p.dim() != 2:
                self.param_groups.pop()
                raise ValueError(f"Muon takes matrices, not a parameter of shape {tuple(p.shape)}")

    def _init_states(self, group, params):
        """Zero state for parameters without one, in flat buffers per device and kind."""
        by_kind = defaultdict(list)
        for p in params:
            by_kind[p.device, group["state_bits"] == 8 and p.numel() >= group["min_8bit_size"]].append(p)
        for (dev, coded), ps in by_kind.items():
            for p, views in zip(ps, _flat_state(dev, [p.shape for p in ps], coded)):
                self.state[p].update(zip(_CODED_KEYS if coded else _BUFFER_KEYS, views))

    @torch.no_grad()
    def step(self, closure=None, *, grad_scale=None):
        loss = None
        if closure is not None:
            with torch.enable_grad():
                loss = closure()
        _check_grad_scale(grad_scale)
        work, fresh = [], []
        for group in self.param_groups:  # checked before any state changes
            live = [p for p in group["params"] if p.grad is not None]
            for p in live:
                if p.grad.is_sparse:
                    raise RuntimeError("Muon does not take sparse gradients")
                if not p.is_contiguous() or not p.grad.is_contiguous():
                    raise RuntimeError("Muon needs contiguous parameters and gradients")
                if not p.is_cuda or p.grad.device != p.device:
                    raise ValueError("Muon needs parameters and gradients on a GPU")
                if not {p.dtype, p.grad.dtype} <= {torch.float32, torch.bfloat16}:
                    raise TypeError("Muon needs float32 or bfloat16 parameters and gradients")
                if grad_scale is not None and grad_scale.device != p.device:
                    raise ValueError("grad_scale must be on the parameters' GPU")
            settings = self._group_settings(group)
            if live:
                _check_settings(**settings)
            new = [p for p in live if not self.state.get(p)]  # without an entry for those that have none
            fresh += new
            work.append((group, live, new, settings))
        if fresh and torch.cuda.is_current_stream_capturing():
            raise RuntimeError("a captured step would begin its state anew in every replay: step once before the capture")
        # every list is made, which is where overlaps are found, before the first one runs
        jobs = []
        try:
            for group, live, new, settings in work:
                self._init_states(group, new)
                batches = {}
                for p in live:
                    st = self.state[p]
                    bits, keys = (8, _CODED_KEYS) if "m_codes" in st else (32, _BUFFER_KEYS)
                    batches.setdefault((p.device, p.dtype, p.grad.dtype, bits), []).append(
                        (p, p.grad, *(st[k] for k in keys)))
                jobs += ((key[-1], _muon_plan(items, key[-1]), settings) for key, items in batches.items())
        except Exception:
            for p in fresh:
                self.state.pop(p, None)
            raise
        for bits, plan, settings in jobs:
            _muon_step(plan, bits, grad_scale, settings)
        return loss

    _params_by_saved_id = Adam8bit._params_by_saved_id

    def _take_state(self, state, groups, keys):
        """Adopt ``state`` (param -> dict) in flat buffers, and ``keys`` of the saved groups."""
        by_kind = defaultdict(list)
        for p, st in state.items():
            by_kind[p.device, "m_codes" in st].append(p)
        for (dev, coded), ps in by_kind.items():
            for p, views in zip(ps, _flat_state(dev, [p.shape for p in ps], coded)):
                for k, t in zip(_CODED_KEYS if coded else _BUFFER_KEYS, views):
                    t.copy_(state[p][k].view(t.shape))
                    state[p][k] = t
        self.state = state
        for group, saved in zip(self.param_groups, groups):
            for k in (saved if keys is None else keys):
                if k != "params":
                    group[k] = saved[k]

    def load_state_dict(self, state_dict):
        """Load a state dict of ``Muon``; each parameter keeps the kind of state that was saved, in
        its own dtypes (torch's loader would cast codes and momentum to the parameter's dtype)."""
        groups = state_dict["param_groups"]
        by_id = self._params_by_saved_id(groups)
        state = defaultdict(dict)
        for pid, st in state_dict["state"].items():
            if not st:  # a parameter that has not been stepped
                continue
            p = by_id[pid]
            n = p.numel()
            want = (("m_codes", torch.uint8, n), ("m_absmax", torch.float32, nblocks(n))) if "m_codes" in st else \
                (("momentum_buffer", torch.float32, n),)
            new = {}
            for k, dt, size in want:
                t = st.get(k)
                if t is None or t.dtype != dt or t.numel() != size:
                    raise ValueError(f"state '{k}' of a parameter with {n} elements must be "
                                     f"{dt} with {size} elements")
                if k == "momentum_buffer" and t.shape != p.shape:
                    raise ValueError("momentum's shape differs from its parameter's")
                new[k] = t.to(device=p.device)
            state[p] = new
        self._take_state(state, groups, None)

    @torch.no_grad()
    def load_fp32_muon_state(self, muon_state_dict):
        """Take over the state of a ``torch.optim.Muon`` state dict with the same parameter groups:
        momenta are quantized block-wise for the parameters that keep codes here and kept in fp32 for
        the others; lr, momentum, weight decay, nesterov, eps and the adjustment are kept.  Other
        Newton-Schulz coefficients than 3.4445, -4.775, 2.0315 have no equivalent here and are refused."""
        groups = [dict(g) for g in muon_state_dict["param_groups"]]
        for g in groups:
            if tuple(g.get("ns_coefficients", (3.4445, -4.775, 2.0315))) != (3.4445, -4.775, 2.0315):
                raise ValueError("other Newton-Schulz coefficients have no equivalent here")
            g["adjust"] = g.get("adjust_lr_fn") or "original"
        by_id = self._params_by_saved_id(groups)
        group_of = {p: g for g in self.param_groups for p in g["params"]}
        state = defaultdict(dict)
        for pid, st in muon_state_dict["state"].items():
            if not st:
                continue
            p = by_id[pid]
            m = st["momentum_buffer"]
            if m.shape != p.shape:
                raise ValueError("momentum's shape differs from its parameter's")
            m = m.to(p.device, torch.float32).contiguous()
            g = group_of[p]
            if g["state_bits"] == 8 and p.numel() >= g["min_8bit_size"]:
                state[p] = dict(zip(_CODED_KEYS, qopt_quantize_blockwise(m.view(-1), SIGNED)))
            else:
                state[p] = {"momentum_buffer": m}
        self._take_state(state, groups, ("lr", "momentum", "weight_decay", "nesterov", "eps", "ns_steps", "adjust"))

    @torch.no_grad()
    def fp32_muon_state_dict(self):
        """A ``torch.optim.Muon``-loadable state dict: every momentum in fp32 and its parameter's
        shape.  (Its loader casts the momenta to the parameter dtype.)"""
        sd = self.state_dict()
        params = [p for g in self.param_groups for p in g["params"]]
        state = {pid: {"momentum_buffer": qopt_dequantize_blockwise(st["m_codes"], st["m_absmax"], SIGNED)
                       .view(params[pid].shape) if "m_codes" in st else st["momentum_buffer"].clone()}
                 for pid, st in sd["state"].items() if st}
        defaults = torch.optim.Muon([torch.zeros(1, 1)]).defaults  # this torch's keys
        groups = [{**defaults, "lr": g["lr"], "momentum": g["momentum"], "weight_decay": g["weight_decay"],
                   "nesterov": g["nesterov"], "eps": g["eps"], "ns_steps": g["ns_steps"],
                   "adjust_lr_fn": g["adjust"], "params": list(g["params"])} for g in sd["param_groups"]]
        return {"state": state, "param_groups": groups}
