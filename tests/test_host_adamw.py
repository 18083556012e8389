"""CPU tests of the AdamW entry points' argument checks (nothing reaches the device) and of
the plan's check that tensors do not overlap."""

import ctypes

import pytest
import torch

qopt = pytest.importorskip("block_wise_bit_adam8bit_amd")
from block_wise_bit_adam8bit_amd import _lib, functional  # noqa: E402


def hparams(**change):
    h = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.1, step=1)
    h.update(change)
    return ctypes.byref(_lib.qopt_adamw_hparams(*h.values()))


def call32(arr, n, pdt=0, gdt=0, hp=None, gs=None):
    return _lib.LIB.qopt_adamw32bit_step(arr, n, pdt, gdt, hparams() if hp is None else hp, gs, None)


def call8(arr, n, pdt=0, gdt=0, hp=None, gs=None, cbm=0x1000, cbv=0x1000):
    return _lib.LIB.qopt_adamw8bit_step(arr, n, pdt, gdt, cbm, cbv, hparams() if hp is None else hp,
                                        gs, None)


T32, T8 = _lib.qopt_tensor32, _lib.qopt_tensor


def one32(p=0x1000, g=0x2000, m=0x3000, v=0x4000, n=10):
    return (T32 * 1)(T32(p, g, m, v, n))


def one8(p=0x1000, g=0x2000, cm=0x3000, cv=0x4000, am=0x5000, av=0x6000, n=10):
    return (T8 * 1)(T8(p, g, cm, cv, am, av, n))


def test_structures():
    assert ctypes.sizeof(T32) == 40
    assert ctypes.sizeof(_lib.qopt_adamw_hparams) == 32


@pytest.mark.parametrize("call,one", [(call32, one32), (call8, one8)])
def test_argument_checks(call, one):
    assert call(None, 0) == qopt.QOPT_OK
    assert call(None, 1) == qopt.QOPT_EINVAL
    assert call(one(), -1) == qopt.QOPT_EINVAL
    assert call(one(), 1, pdt=2) == qopt.QOPT_EUNSUPPORTED
    assert call(one(), 1, gdt=-1) == qopt.QOPT_EUNSUPPORTED
    assert call(one(n=-1), 1) == qopt.QOPT_EINVAL
    assert call(one(p=0, n=0), 1) == qopt.QOPT_OK
    for name in ("p", "g"):
        assert call(one(**{name: 0}), 1) == qopt.QOPT_EINVAL
        assert call(one(**{name: 0x1002}), 1) == qopt.QOPT_EALIGN
        assert call(one(**{name: 0x1001}), 1, pdt=1, gdt=1) == qopt.QOPT_EALIGN
    assert call(one(), 1, gs=0x1002) == qopt.QOPT_EALIGN
    for change in (dict(step=0), dict(beta1=1.0), dict(beta2=-0.1), dict(eps=-1.0),
                   dict(lr=float("inf")), dict(eps=float("nan")), dict(weight_decay=-1e-3),
                   dict(weight_decay=float("inf")), dict(weight_decay=float("nan"))):
        assert call(one(), 1, hp=hparams(**change)) == qopt.QOPT_EINVAL, change


def test_null_and_misaligned_state():
    for name in ("m", "v"):
        assert call32(one32(**{name: 0}), 1) == qopt.QOPT_EINVAL
        assert call32(one32(**{name: 0x1002}), 1) == qopt.QOPT_EALIGN
    for name in ("cm", "cv", "am", "av"):
        assert call8(one8(**{name: 0}), 1) == qopt.QOPT_EINVAL
    assert call8(one8(am=0x1002), 1) == qopt.QOPT_EALIGN
    assert call8(one8(), 1, cbm=None) == qopt.QOPT_EINVAL
    assert call8(one8(), 1, cbv=0x1008) == qopt.QOPT_EALIGN
    assert _lib.LIB.qopt_adamw32bit_step(one32(), 1, 0, 0, None, None, None) == qopt.QOPT_EINVAL
    assert _lib.LIB.qopt_adamw8bit_step(one8(), 1, 0, 0, 0x1000, 0x1000, None, None,
                                        None) == qopt.QOPT_EINVAL


def test_overlap_check():
    import torch
    a, b, c, d = (torch.zeros(100) for _ in range(4))
    def check(tensors):
        functional._check_spans([(x.data_ptr(), x.data_ptr() + x.numel() * x.element_size(), i != 1)
                                 for t in tensors for i, x in enumerate(t) if x.numel()])

    check([(a, b, c, d)])
    check([(a[:50], b, c[:50], d[:50]), (a[50:], b, c[50:], d[50:])])  # a gradient serves two
    check([(a[:0], a[:0], a[:0], a[:0]), (a, b, c, d)])
    for bad in ([(a, a, c, d)], [(a, b, c, c)], [(a, b[10:], c, b[:11])],
                [(a, b, c, d), (a[99:], b[:1], torch.zeros(1), torch.zeros(1))]):
        with pytest.raises(ValueError):
            check(bad)


def test_optimizer_refuses_cpu_parameters():
    p = torch.nn.Parameter(torch.ones(8192))
    p.grad = torch.ones(8192)
    opt = qopt.AdamW([p])
    with pytest.raises(ValueError):
        opt.step()
    assert not any(opt.state.values())


def test_optimizer_looks_at_grad_scale_first():
    """Before any parameter, and so before any state exists: its type and its size."""
    p = torch.nn.Parameter(torch.ones(8192))
    p.grad = torch.ones(8192)
    opt = qopt.AdamW([p])
    for bad in (torch.ones(2), torch.ones(0), torch.ones(1, dtype=torch.float64), torch.ones(1, dtype=torch.bfloat16)):
        with pytest.raises(ValueError, match="grad_scale must be one float32"):
            opt.step(grad_scale=bad)
    assert not any(opt.state.values())
