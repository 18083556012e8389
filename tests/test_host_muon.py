"""CPU tests of the Muon entry points' argument checks: nothing reaches the device."""

import ctypes

import pytest
import torch

qopt = pytest.importorskip("block_wise_bit_adam8bit_amd")
from block_wise_bit_adam8bit_amd import _lib  # noqa: E402

L = _lib.LIB
OK, EINVAL, EUNSUPPORTED, EALIGN = qopt.QOPT_OK, qopt.QOPT_EINVAL, qopt.QOPT_EUNSUPPORTED, qopt.QOPT_EALIGN
P = 0x1000  # a stand-in address: every check fails, or has nothing to do, before its use
MOST = _lib.QOPT_MUON_MAX_DIM


def test_header_mirror():
    c = _lib.header_constants()
    assert c["QOPT_MUON_MAX_DIM"] == MOST and c["QOPT_MUON_MAX_STEPS"] == _lib.QOPT_MUON_MAX_STEPS


def test_orthogonalize_checks():
    def call(x=P, dt=0, batch=1, rows=8, cols=8, steps=5, eps=1e-7, out=P, odt=0, ws=P, nws=1 << 40):
        return L.qopt_orthogonalize(x, dt, batch, rows, cols, steps, eps, out, odt, ws, nws, None)

    assert call(batch=0) == OK and call(rows=0, x=None) == OK and call(cols=0, out=None, ws=None, nws=0) == OK
    n = ctypes.c_size_t(0)
    assert L.qopt_orthogonalize_workspace(1, 8, 8, ctypes.byref(n)) == OK and n.value > 0
    for bad in (dict(batch=-1), dict(rows=-1), dict(cols=-1), dict(rows=MOST + 1), dict(cols=MOST + 1), dict(steps=0),
                dict(steps=_lib.QOPT_MUON_MAX_STEPS + 1), dict(eps=0.0), dict(eps=-1.0), dict(eps=float("nan")),
                dict(eps=float("inf")), dict(x=None), dict(out=None), dict(ws=None), dict(nws=n.value - 1)):
        assert call(**bad) == EINVAL, bad
    for bad in (dict(dt=2), dict(odt=-1)):
        assert call(**bad) == EUNSUPPORTED, bad
    for bad in (dict(x=P + 2), dict(x=P + 1, dt=1), dict(out=P + 2), dict(ws=P + 128)):
        assert call(**bad) == EALIGN, bad


def hparams(lr=1e-3, momentum=0.95, wd=0.1, eps=1e-7, nesterov=1, adjust=0, steps=5):
    return ctypes.byref(_lib.qopt_muon_hparams(lr, momentum, wd, eps, nesterov, adjust, steps))


def tensors(*items):
    return (_lib.qopt_muon_tensor * len(items))(*items)


@pytest.mark.parametrize("bits", [8, 32])
def test_step_checks(bits):
    step = getattr(L, f"qopt_muon{bits}bit_step")

    def call(param=P, grad=P, m=P, am=P, rows=8, cols=8, n=1, pdt=0, gdt=0, cb=P, gs=None, ws=P, nws=1 << 40, hp=None, **h):
        arr = tensors((param, grad, m, am, rows, cols)) if n else None
        return step(arr, n, pdt, gdt, *((cb,) if bits == 8 else ()), hp or hparams(**h), gs, ws, nws, None)

    assert call(n=0) == OK and call(rows=0, param=None, grad=None, m=None, am=None, ws=None, nws=0) == OK
    need = ctypes.c_size_t(0)
    assert L.qopt_muon_workspace(tensors((P, P, P, P, 8, 8)), 1, ctypes.byref(need)) == OK and need.value > 0
    inf, nan = float("inf"), float("nan")
    for bad in (dict(lr=-1.0), dict(lr=inf), dict(lr=nan), dict(momentum=1.0), dict(momentum=-0.1), dict(momentum=nan),
                dict(wd=-0.1), dict(wd=nan), dict(eps=0.0), dict(eps=inf), dict(nesterov=2), dict(steps=0),
                dict(steps=1000)):
        assert call(**bad) == EINVAL and call(n=0, **bad) == EINVAL, bad
    for bad in (dict(param=None), dict(grad=None), dict(m=None), dict(rows=-1), dict(cols=MOST + 1), dict(ws=None),
                dict(nws=need.value - 1)) + ((dict(am=None), dict(cb=None)) if bits == 8 else ()):
        assert call(**bad) == EINVAL, bad
    assert step(None, 1, 0, 0, *((P,) if bits == 8 else ()), hparams(), None, P, 1 << 40, None) == EINVAL
    assert step(None, -1, 0, 0, *((P,) if bits == 8 else ()), hparams(), None, P, 1 << 40, None) == EINVAL
    assert step(None, 0, 0, 0, *((P,) if bits == 8 else ()), None, None, P, 1 << 40, None) == EINVAL
    for bad in (dict(pdt=2), dict(gdt=-1), dict(adjust=2), dict(adjust=-1)):
        assert call(**bad) == EUNSUPPORTED, bad
    for bad in (dict(param=P + 2), dict(grad=P + 1), dict(gs=P + 2), dict(ws=P + 16)) + \
            ((dict(am=P + 2), dict(cb=P + 8)) if bits == 8 else (dict(m=P + 2),)):
        assert call(**bad) == EALIGN, bad


def test_workspace_queries():
    n = ctypes.c_size_t(7)
    q = L.qopt_orthogonalize_workspace
    assert q(0, 64, 64, ctypes.byref(n)) == OK and n.value == 0
    assert q(4, 0, 64, ctypes.byref(n)) == OK and n.value == 0
    assert q(4, 4, 4, None) == EINVAL and q(-1, 4, 4, ctypes.byref(n)) == EINVAL and q(1, MOST + 1, 4, ctypes.byref(n)) == EINVAL
    assert q(1, 100, 300, ctypes.byref(n)) == OK
    one = n.value
    assert q(1, 300, 100, ctypes.byref(n)) == OK and n.value == one
    assert q(1000, 100, 300, ctypes.byref(n)) == OK and n.value <= 33 * one  # lots are bounded
    assert L.qopt_muon_workspace(tensors((0, 0, 0, 0, 100, 300), (0, 0, 0, 0, 0, 5)), 2, ctypes.byref(n)) == OK and n.value == one
    assert L.qopt_muon_workspace(None, 0, ctypes.byref(n)) == OK and n.value == 0
    assert L.qopt_muon_workspace(None, 1, ctypes.byref(n)) == EINVAL and L.qopt_muon_workspace(None, 0, None) == EINVAL


@pytest.mark.parametrize("batch,rows,cols", [
    (47, 311, 1713), (79, 856, 1029), (44, 1593, 270), (62, 1689, 325), (63, 747, 2144), (77, 1548, 311),  # smaller last lots ask for more
    (1, 64, 64), (16, 200, 300), (17, 200, 300), (32, 100, 100), (33, 100, 100), (33, 20, 4000), (65, 32, 33), (5, 2048, 2048)])
def test_a_batch_asks_for_what_its_matrices_one_by_one_do(batch, rows, cols):
    one, each = ctypes.c_size_t(0), ctypes.c_size_t(0)
    assert L.qopt_orthogonalize_workspace(batch, rows, cols, ctypes.byref(one)) == OK
    assert L.qopt_muon_workspace(tensors(*[(0, 0, 0, 0, rows, cols)] * batch), batch, ctypes.byref(each)) == OK
    assert one.value == each.value


def test_wrappers_refuse():
    x = torch.zeros(4, 8)
    codes, am = torch.zeros(32, dtype=torch.uint8), torch.zeros(1)
    hp = dict(lr=1e-3, momentum=0.9, weight_decay=0.0)
    for err, call in (
            (ValueError, lambda: qopt.qopt_orthogonalize(x)),  # on the CPU
            (ValueError, lambda: qopt.qopt_muon8bit_plan([(x, x.clone(), codes, am)])),
            (TypeError, lambda: qopt.qopt_orthogonalize(x.half())),
            (TypeError, lambda: qopt.qopt_orthogonalize(x, out_dtype=torch.float16)),
            (ValueError, lambda: qopt.qopt_orthogonalize(x[0])),
            (ValueError, lambda: qopt.qopt_orthogonalize(x.t())),
            (ValueError, lambda: qopt.qopt_orthogonalize(x, steps=0)),
            (ValueError, lambda: qopt.qopt_orthogonalize(x, steps=2.5)),
            (ValueError, lambda: qopt.qopt_orthogonalize(x, eps=0.0)),
            (ValueError, lambda: qopt.qopt_muon8bit_plan([(x, x.clone(), codes)])),
            (ValueError, lambda: qopt.qopt_muon32bit_plan([(x, x.clone(), codes, am)])),
            (ValueError, lambda: qopt.qopt_muon32bit_plan([(x[0], x[0].clone(), x[0].clone())])),
            (ValueError, lambda: qopt.qopt_muon32bit_plan([(x, x.t(), x.clone())])),
            (ValueError, lambda: qopt.qopt_muon32bit_plan([(x, x.clone(), am)])),
            (TypeError, lambda: qopt.qopt_muon32bit_plan([(x, x.clone(), x.bfloat16())])),
            (TypeError, lambda: qopt.qopt_muon32bit_plan([(x.double(), x.clone(), x.clone())])),
            (TypeError, lambda: qopt.qopt_muon8bit_plan([(x, x.clone(), codes.int(), am)])),
            (ValueError, lambda: qopt.qopt_muon8bit_plan([(x, x.clone(), codes, am.repeat(2))])),
            (ValueError, lambda: qopt.qopt_muon32bit_step([], **hp, adjust="other")),
            (ValueError, lambda: qopt.qopt_muon32bit_step([], **hp, steps=99)),
            (ValueError, lambda: qopt.qopt_muon32bit_step([], **hp, grad_scale=torch.zeros(2))),
            (qopt.QoptError, lambda: qopt.qopt_muon32bit_step([], **{**hp, "lr": -1.0}))):
        with pytest.raises(err):
            call()
    qopt.qopt_muon32bit_step([], **hp)
    with pytest.raises(ValueError):
        qopt.qopt_muon8bit_step(qopt.qopt_muon32bit_plan([]), **hp)


def test_optimizer_checks():
    p = torch.nn.Parameter(torch.zeros(4, 4))
    for bad in (dict(lr=-1.0), dict(momentum=1.0), dict(weight_decay=-0.1), dict(state_bits=16), dict(adjust="x"),
                dict(ns_steps=0), dict(eps=0.0)):
        with pytest.raises(ValueError):
            qopt.Muon([p], **bad)
    with pytest.raises(ValueError):
        qopt.Muon([p, torch.nn.Parameter(torch.zeros(4))])
    opt = qopt.Muon([p])
    with pytest.raises(ValueError):
        opt.add_param_group(dict(params=[torch.nn.Parameter(torch.zeros(2, 2, 2))]))
    assert len(opt.param_groups) == 1
    p.grad = torch.zeros(4, 4)
    with pytest.raises(ValueError):  # on the CPU
        opt.step()
    assert not opt.state
