"""CPU pins of the AdamW oracle: against the Adam oracle where the two coincide, against
torch.optim.AdamW in binary64 over many steps, and against closed forms."""

import numpy as np
import pytest
import torch

import oracle
from oracle import BLOCK

HP = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8)


def state(n):
    nb = -(-n // BLOCK)
    return [np.zeros(n, np.uint8), np.zeros(n, np.uint8), np.zeros(nb, np.float32),
            np.zeros(nb, np.float32)]


@pytest.mark.parametrize("pdt,gdt", [("f32", "f32"), ("f32", "bf16"), ("bf16", "f32"),
                                     ("bf16", "bf16")])
def test_without_decay_and_factor_it_is_adam(pdt, gdt):
    rng = np.random.default_rng(3)
    n = 3 * BLOCK + 5
    p = rng.normal(0, 0.02, n).astype(np.float32)
    p = oracle.f32_to_bf16_rne(p) if pdt == "bf16" else p
    a = b = (p, *state(n))
    for step in range(1, 5):
        g = rng.normal(0, 1e-3, n).astype(np.float32)
        g = oracle.f32_to_bf16_rne(g) if gdt == "bf16" else g
        kw = dict(step=step, param_dtype=pdt, grad_dtype=gdt, **HP)
        a = oracle.adam8bit_step(a[0], g, *a[1:], **kw)
        b = oracle.adamw8bit_step(b[0], g, *b[1:], weight_decay=0.0, grad_scale=1.0, **kw)
        for x, y in zip(a, b):
            assert np.array_equal(x, y)


def test_32_bit_moments_follow_torch_in_binary64():
    # Each step the parameter's update is at most lr (1 + a few ulps) in size here and its
    # binary32 evaluation is off by under 12 roundings of its own size plus 2 of the
    # parameter's: |dp| per step <= 2^-24 (12 lr + 2 |p|).  The moments' own rounding errors
    # (under 2^-22 relative per step, decaying) move the update by under 2^-20 lr.
    rng = np.random.default_rng(5)
    n, steps, wd = 4001, 40, 0.1
    p = rng.normal(0, 0.02, n).astype(np.float32)
    m = np.zeros(n, np.float32)
    v = np.zeros(n, np.float32)
    f = lambda x: float(np.float32(x))  # noqa: E731
    t = torch.nn.Parameter(torch.from_numpy(p.astype(np.float64)))
    opt = torch.optim.AdamW([t], lr=f(HP["lr"]), betas=(f(HP["beta1"]), f(HP["beta2"])),
                            eps=f(HP["eps"]), weight_decay=f(wd))
    for step in range(1, steps + 1):
        g = rng.normal(0, 1e-3, n).astype(np.float32)
        p, m, v = oracle.adamw32bit_step(p, g, m, v, weight_decay=wd, step=step, grad_scale=0.5,
                                         **HP)
        t.grad = torch.from_numpy(g.astype(np.float64) * 0.5)
        opt.step()
    ref = t.detach().numpy()
    bound = steps * (2.0 ** -24 * (12 * HP["lr"] + 2 * (np.abs(ref) + steps * HP["lr"]))
                     + 2.0 ** -20 * HP["lr"])
    assert np.all(np.abs(p - ref) <= bound)
    for got, key in ((m, "exp_avg"), (v, "exp_avg_sq")):
        want = opt.state[t][key].numpy()
        # every term of the sum carries under 4 roundings a step, all of them decaying
        size = np.abs(want) + np.abs(want).max()
        assert np.all(np.abs(got - want) <= 2.0 ** -24 * 4 * steps * size)


def test_decay_and_factor_closed_forms():
    # a zero gradient leaves only the decay: p' = p * fl32(1 - lr wd)
    n = BLOCK
    p = np.linspace(-1, 1, n).astype(np.float32)
    out = oracle.adamw8bit_step(p, np.zeros(n, np.float32), *state(n), weight_decay=0.25, step=1,
                                lr=0.5, beta1=0.9, beta2=0.999, eps=1e-8)
    assert np.array_equal(out[0], p * np.float32(0.875))
    assert oracle.decay_factor(0.5, 0.25) == np.float32(0.875)
    # a power-of-two factor scales m by itself and v by its square, exactly
    rng = np.random.default_rng(1)
    g = rng.normal(0, 1, n).astype(np.float32)
    z = np.zeros(n, np.float32)
    kw = dict(weight_decay=0.0, step=1, **HP)
    a = oracle.adamw32bit_step(p, g, z, z, **kw)
    b = oracle.adamw32bit_step(p, g, z, z, grad_scale=0.25, **kw)
    assert np.array_equal(b[1], a[1] * np.float32(0.25))
    assert np.array_equal(b[2], a[2] * np.float32(0.0625))
