"""GPU test of the workspaces: what the queries ask for is all that is written."""

import ctypes

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
BEHIND = 320 << 20  # bytes watched behind a workspace: more than twice all partial sums of a launch


@pytest.fixture(scope="module")
def q():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import block_wise_bit_adam8bit_amd as q
    torch.cuda.set_device(0)
    return q


def watched(need):
    buf = torch.empty(need + BEHIND, dtype=torch.uint8, device="cuda")
    buf[need:].fill_(0xA5)
    return buf


def shapes(seed, count, most):
    rng = np.random.default_rng(seed)
    return [tuple(int(v) for v in np.exp(rng.uniform(0, np.log(most), 2)).round()) for _ in range(count)]


@pytest.mark.parametrize("seed", range(4))
def test_a_batch_stays_in_its_workspace(q, seed):
    """Batches that end in smaller lots among them."""
    rng = np.random.default_rng(seed)
    cases = [(int(rng.integers(1, 50)), r, c) for r, c in shapes(seed, 8, 1500)]
    cases += [[(47, 311, 1713)], [(44, 1593, 270)], [(17, 200, 300)], [(1, 4096, 4096), (5, 2048, 300)]][seed]
    for batch, rows, cols in cases:
        for out in (torch.float32, torch.bfloat16):
            print(f"orthogonalize {batch}x{rows}x{cols} {out}", flush=True)
            x = torch.randn(batch, rows, cols, device="cuda")
            y = torch.empty_like(x, dtype=out)
            need = ctypes.c_size_t(0)
            assert q.LIB.qopt_orthogonalize_workspace(batch, rows, cols, ctypes.byref(need)) == q.QOPT_OK
            ws = watched(need.value)
            assert q.LIB.qopt_orthogonalize(x.data_ptr(), 0, batch, rows, cols, 5, 1e-7, y.data_ptr(),
                                            1 if out is torch.bfloat16 else 0, ws.data_ptr(), need.value,
                                            torch.cuda.current_stream().cuda_stream) == q.QOPT_OK
            assert bool((ws[need.value:] == 0xA5).all())
            assert torch.equal(y, q.qopt_orthogonalize(x, out_dtype=out))
            del x, y, ws


@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("seed", range(3))
def test_a_step_stays_in_its_workspace(q, seed, bits):
    from block_wise_bit_adam8bit_amd import _lib
    sizes = shapes(100 + seed, 30, 1800) + [(2048, 2048), (64, 20000)]
    for dtype in (torch.float32, torch.bfloat16):
        print(f"muon {bits} bits {dtype} {sizes}", flush=True)
        items = []
        for r, c in sizes:
            p, g = torch.zeros(r, c, dtype=dtype, device="cuda"), torch.randn(r, c, device="cuda")
            state = (torch.zeros(r, c, device="cuda"),) if bits == 32 else \
                (torch.zeros(r * c, dtype=torch.uint8, device="cuda"), torch.zeros(-(-r * c // 2048), device="cuda"))
            items.append((p, g, *state))
        plan = (q.qopt_muon8bit_plan if bits == 8 else q.qopt_muon32bit_plan)(items)
        ws = watched(plan.room)
        hp = _lib.qopt_muon_hparams(0.1, 0.9, 0.0, 1e-7, 1, 0, 5)
        args = (plan.array, len(plan.array), plan.pdtype, plan.gdtype) + \
            ((q.codebook(q.SIGNED, plan.device).data_ptr(),) if bits == 8 else ()) + \
            (ctypes.byref(hp), None, ws.data_ptr(), plan.room, torch.cuda.current_stream().cuda_stream)
        assert getattr(q.LIB, f"qopt_muon{bits}bit_step")(*args) == q.QOPT_OK
        assert bool((ws[plan.room:] == 0xA5).all())
        got = [t[0].clone() for t in items]
        for t in items:
            for x in (t[0], *t[2:]):
                x.zero_()
        (q.qopt_muon8bit_step if bits == 8 else q.qopt_muon32bit_step)(plan, lr=0.1, momentum=0.9, weight_decay=0.0)
        assert all(torch.equal(a, t[0]) for a, t in zip(got, items))
