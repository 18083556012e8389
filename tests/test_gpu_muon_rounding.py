"""GPU tests of what a bfloat16 destination of the orthogonalisation loses: its own rounding and nothing else
that binary32 would keep.

A result y rounded to bfloat16 from some z has |y - z| at most half of the spacing at y, so what |y - want|
exceeds that half by is at most |z - want|, place by place.  In the Frobenius norm that excess is therefore
bounded as a binary32 result is (``result_bound``: 8 times what rounding every stored value to 22 bits moves the matrix by, and
as much again for binary32 sums of k terms, sqrt(k) / 2 roundings of 2^-24 or sqrt(k) / 8 of 2^-22).  Half of the
spacing itself is not in the bound, so that 11 or 15 bits in place of 22 do not pass."""

import numpy as np
import pytest
import torch

from oracle import muon

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module")
def q():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import block_wise_bit_adam8bit_amd as q
    torch.cuda.set_device(0)
    return q


def host(t):
    return t.detach().double().cpu().numpy()


def gradient(rng, rows, cols, kind):
    u = rng.normal(size=(rows, cols)) * 1e-3
    if kind == "steep":  # a few directions hold nearly everything
        r = min(3, rows, cols)
        u = u * 0.05 + rng.normal(size=(rows, r)) @ rng.normal(size=(r, cols)) * 2e-3
    if kind == "spike":  # one entry does
        u[rows // 2, cols // 3] = 1.0
    return u.astype(np.float32)


@pytest.mark.parametrize("kind", ["normal", "steep", "spike"])
@pytest.mark.parametrize("rows,cols", [(33, 40), (64, 64), (65, 130), (300, 99), (128, 129), (200, 1000), (257, 256), (600, 700),
                                       (1000, 40), (900, 820)])
def test_one_rounding_to_bf16(q, rows, cols, kind):
    print(f"orthogonalize {rows}x{cols} {kind}", flush=True)
    x = gradient(np.random.default_rng(rows * 1000 + cols), rows, cols, kind)
    for src in (F32, BF16):
        u = torch.from_numpy(x).to("cuda", src)
        want, most = muon.result_bound(host(u))
        off = np.linalg.norm(muon.beyond_half(host(q.qopt_orthogonalize(u, out_dtype=BF16)), want))
        assert off <= most, (src, off, most, off / np.linalg.norm(want))


@pytest.mark.parametrize("steps", [1, 2, 3, 4, 6, 8, 9])
def test_one_rounding_after_other_numbers_of_iterations(q, steps):
    rng = np.random.default_rng(steps)
    for rows, cols in ((70, 200), (200, 70)):
        u = torch.from_numpy(gradient(rng, rows, cols, "normal")).cuda()
        want, most = muon.result_bound(host(u), steps)
        off = np.linalg.norm(muon.beyond_half(host(q.qopt_orthogonalize(u, steps=steps, out_dtype=BF16)), want))
        assert off <= most, (off, most)


@pytest.mark.parametrize("batch,rows,cols", [(4, 2048, 2048), (1, 1500, 4200), (1, 4400, 1200), (1, 129, 20000)])
def test_one_rounding_of_large_matrices(q, batch, rows, cols):
    """The iterations of a shorter side above 768 are grouped alike for either destination, so the bfloat16 result is the
    binary32 one rounded; below, the groups' lengths differ, and the two differ by what a binary32 result may be off."""
    print(f"orthogonalize {batch}x{rows}x{cols}", flush=True)
    g = torch.Generator(device="cuda").manual_seed(rows)
    x = torch.randn(batch, rows, cols, generator=g, device="cuda") * 1e-3
    y, z = (q.qopt_orthogonalize(x, out_dtype=dt) for dt in (BF16, F32))
    if min(rows, cols) > 768:
        assert torch.equal(y, z.to(BF16))
    else:
        # 3e-7 is what rounding to 22 bits moves normal matrices by
        most = 2 * 8 * 3e-7 * (1 + max(rows, cols) ** 0.5 / 8) * np.linalg.norm(host(z))
        assert np.linalg.norm(muon.beyond_half(host(y), host(z))) <= most


@pytest.mark.parametrize("bits", [8, 32])
def test_one_rounding_of_a_bf16_parameter(q, bits):
    """A step with nothing but the update: no decay, momentum 0, parameters of zeros, so that they become -rate O(g) rounded once
    (and rate O(g) once in binary32, where it is off by 2^-24 of itself, besides the product's)."""
    rng = np.random.default_rng(bits)
    ts = []
    for rows, cols in ((96, 200), (200, 96), (800, 780)):
        g = torch.from_numpy(gradient(rng, rows, cols, "normal")).cuda()
        m = torch.zeros(rows, cols, device="cuda") if bits == 32 else torch.zeros(rows * cols, dtype=torch.uint8, device="cuda")
        am = () if bits == 32 else (torch.zeros(-(-rows * cols // 2048), device="cuda"),)
        ts.append((torch.zeros(rows, cols, dtype=BF16, device="cuda"), g, m, *am))
    step = q.qopt_muon8bit_step if bits == 8 else q.qopt_muon32bit_step
    step(ts, lr=0.5, momentum=0.0, weight_decay=0.0, nesterov=False)
    for p, g, *_ in ts:
        want, most = muon.result_bound(host(g))
        r = float(muon.rate(0.5, *p.shape, "original"))
        off = np.linalg.norm(muon.beyond_half(host(p), -r * want))
        assert off <= r * (most + 2 * 2.0 ** -24 * np.linalg.norm(want)), (p.shape, off, most)
