"""Oracle: AdamW steps, with 8-bit and with 32-bit moments (test infrastructure only).

AdamW is Adam with the weight decay taken out of the gradient and applied to the
parameter (Loshchilov and Hutter, "Decoupled Weight Decay Regularization").  Readings:

* decay = fl32(1 - lr * wd), evaluated in binary64 from binary32 lr and wd; the parameter
  is multiplied with it first, in binary32, and the Adam update of ``adam8bit.py`` then
  starts from the product.  bf16 parameters are rounded once, after the update.
* gradients are multiplied with an optional binary32 factor first, in binary32.
* with 32-bit moments the arithmetic is the same, and the moments are stored as computed.
"""

import numpy as np

from .adam8bit import adam8bit_step, adam_scalars, bf16_to_f32, f32_to_bf16_rne

F32 = np.float32


def decay_factor(lr, weight_decay):
    return F32(1.0 - float(F32(lr)) * float(F32(weight_decay)))


def _prepared(p, g, lr, weight_decay, grad_scale, param_dtype, grad_dtype):
    p32 = bf16_to_f32(p) if param_dtype == "bf16" else np.asarray(p, dtype=F32)
    g32 = bf16_to_f32(g) if grad_dtype == "bf16" else np.asarray(g, dtype=F32)
    if grad_scale is not None:
        g32 = g32 * F32(grad_scale)
    return p32.reshape(-1) * decay_factor(lr, weight_decay), g32.reshape(-1)


def adamw8bit_step(p, g, cm, cv, am, av, *, lr, beta1, beta2, eps, weight_decay, step,
                   grad_scale=None, param_dtype="f32", grad_dtype="f32"):
    """One 8-bit AdamW step on one tensor, laid out as ``adam8bit_step``.
    Parity: pinned (equals adam8bit_step without decay and factor; the decayed parameter and
    the scaled gradient against their closed forms)."""
    p32, g32 = _prepared(p, g, lr, weight_decay, grad_scale, param_dtype, grad_dtype)
    out = adam8bit_step(p32, g32, cm, cv, am, av, lr=lr, beta1=beta1, beta2=beta2, eps=eps,
                        step=step)
    return (f32_to_bf16_rne(out[0]) if param_dtype == "bf16" else out[0], *out[1:])


def adamw32bit_step(p, g, m, v, *, lr, beta1, beta2, eps, weight_decay, step, grad_scale=None,
                    param_dtype="f32", grad_dtype="f32"):
    """One AdamW step with fp32 moments on one tensor; returns (p', m', v').
    Parity: pinned (against torch.optim.AdamW in binary64 over many steps, within its
    rounding bound)."""
    b1, b2, omb1, omb2, eps32, step_size, inv_sqrt_bc2 = adam_scalars(lr, beta1, beta2, eps, step)
    p32, g32 = _prepared(p, g, lr, weight_decay, grad_scale, param_dtype, grad_dtype)
    m = (b1 * np.asarray(m, F32)) + (omb1 * g32)
    v = (b2 * np.asarray(v, F32)) + (omb2 * (g32 * g32))
    denom = (np.sqrt(v) * inv_sqrt_bc2) + eps32
    out = p32 - (step_size * (m / denom))
    return (f32_to_bf16_rne(out) if param_dtype == "bf16" else out), m, v
