"""CPU tests of the layer normalisation's argument checks: nothing reaches the device."""

import ctypes

import pytest
import torch

qopt = pytest.importorskip("block_wise_bit_adam8bit_amd")
from block_wise_bit_adam8bit_amd import _lib  # noqa: E402

L = _lib.LIB
OK, EINVAL, EUNSUPPORTED, EALIGN = qopt.QOPT_OK, qopt.QOPT_EINVAL, qopt.QOPT_EUNSUPPORTED, qopt.QOPT_EALIGN
P = 0x1000  # a stand-in address: every check fails, or has nothing to do, before its use


def test_header_mirror():
    c = _lib.header_constants()
    assert c["QOPT_NORM_MAX_DIM"] == _lib.QOPT_NORM_MAX_DIM
    assert c["QOPT_NORM_MAX_ROWS"] == _lib.QOPT_NORM_MAX_ROWS


def test_forward_checks():
    def call(x=P, dt=1, rows=4, dim=8, ldx=8, w=P, b=P, wdt=0, eps=1e-5, out=P, ldo=8, mean=P, rstd=P):
        return L.qopt_layer_norm_forward(x, dt, rows, dim, ldx, w, b, wdt, eps, out, ldo, mean, rstd, None)

    assert call(rows=0) == OK and call(rows=0, x=None, out=None) == OK and call(dim=0, ldx=0, ldo=0) == OK
    for bad in (dict(rows=-1), dict(dim=-1), dict(ldx=7), dict(ldo=7), dict(x=None), dict(out=None),
                dict(eps=-1e-5), dict(eps=float("nan")), dict(eps=float("inf")),
                dict(rows=_lib.QOPT_NORM_MAX_ROWS + 1), dict(dim=_lib.QOPT_NORM_MAX_DIM + 1, ldx=1 << 30, ldo=1 << 30),
                dict(ldx=1 << 62), dict(ldo=1 << 62)):
        assert call(**bad) == EINVAL, bad
    for bad in (dict(dt=2), dict(dt=-1), dict(wdt=2), dict(wdt=-1)):
        assert call(**bad) == EUNSUPPORTED, bad
    for bad in (dict(x=P + 1), dict(x=P + 2, dt=0), dict(out=P + 1), dict(w=P + 2), dict(b=P + 1, wdt=1),
                dict(mean=P + 2), dict(rstd=P + 1)):
        assert call(**bad) == EALIGN, bad


def test_backward_checks():
    def call(x=P, dt=1, rows=4, dim=8, ldx=8, w=P, wdt=0, mean=P, rstd=P, g=P, ldg=8, dx=P, lddx=8, dw=P, db=P,
             ws=P, nws=1 << 20):
        return L.qopt_layer_norm_backward(x, dt, rows, dim, ldx, w, wdt, mean, rstd, g, ldg, dx, lddx, dw, db, ws,
                                          nws, None)

    assert call(dim=0, ldx=0, ldg=0, lddx=0) == OK
    assert call(rows=0, dw=None, db=None, x=None, g=None, mean=None, rstd=None) == OK
    assert call(rows=0, dw=None, db=None, dx=None, ws=None, nws=0) == OK
    for bad in (dict(rows=-1), dict(dim=-1), dict(ldx=7), dict(ldg=7), dict(lddx=7), dict(x=None), dict(g=None),
                dict(mean=None), dict(rstd=None), dict(ws=None), dict(nws=63)):
        assert call(**bad) == EINVAL, bad
    for bad in (dict(dt=2), dict(wdt=7)):
        assert call(**bad) == EUNSUPPORTED, bad
    for bad in (dict(x=P + 1), dict(g=P + 1), dict(dx=P + 1), dict(w=P + 2), dict(dw=P + 2), dict(db=P + 2),
                dict(mean=P + 2), dict(rstd=P + 2), dict(ws=P + 8)):
        assert call(**bad) == EALIGN, bad


def test_workspace_query():
    n = ctypes.c_size_t(7)
    q = L.qopt_layer_norm_backward_workspace
    assert q(0, 64, ctypes.byref(n)) == OK and n.value == 0
    assert q(1, 64, ctypes.byref(n)) == OK and n.value == 2 * 64 * 4
    assert q(1 << 30, 64, ctypes.byref(n)) == OK and n.value <= 1 << 20
    assert q(4, 4, None) == EINVAL and q(-1, 4, ctypes.byref(n)) == EINVAL
    assert q(4, _lib.QOPT_NORM_MAX_DIM + 1, ctypes.byref(n)) == EINVAL


def test_wrappers_refuse():
    x, w = torch.zeros(4, 8), torch.ones(8)
    stats = torch.zeros(4)
    for err, call in (
            (ValueError, lambda: qopt.layer_norm(x, w, w)),  # on the CPU
            (ValueError, lambda: qopt.qopt_layer_norm_forward(x, w, w)),
            (ValueError, lambda: qopt.qopt_layer_norm_backward(x, w, stats, stats, x)),
            (TypeError, lambda: qopt.layer_norm(x.half())),
            (TypeError, lambda: qopt.layer_norm(x, w.half())),
            (TypeError, lambda: qopt.layer_norm(x, w, w.bfloat16())),
            (TypeError, lambda: qopt.qopt_layer_norm_forward(x, w, w.bfloat16())),
            (ValueError, lambda: qopt.layer_norm(x, w[:7])),
            (ValueError, lambda: qopt.layer_norm(x, None, w[None])),
            (ValueError, lambda: qopt.layer_norm(x[0, 0])),
            (ValueError, lambda: qopt.qopt_layer_norm_forward(x, w, eps=-1.0)),
            (ValueError, lambda: qopt.qopt_layer_norm_forward(x, w, eps=float("nan"))),
            (ValueError, lambda: qopt.qopt_layer_norm_forward(x.t().contiguous().t(), w)),
            (ValueError, lambda: qopt.qopt_layer_norm_forward(x[:1].expand(4, 8), w)),
            (ValueError, lambda: qopt.qopt_layer_norm_forward(x.view(2, 2, 8).transpose(0, 1), w)),
            (ValueError, lambda: qopt.qopt_layer_norm_backward(x, w, stats, stats, x[:3])),
            (ValueError, lambda: qopt.qopt_layer_norm_backward(x, w, stats, stats, x.bfloat16())),
            (ValueError, lambda: qopt.qopt_layer_norm_backward(x, w, stats[:3], stats, x)),
            (ValueError, lambda: qopt.qopt_layer_norm_backward(x, w, stats, stats.double(), x)),
            (TypeError, lambda: qopt.qopt_layer_norm_backward(x, w, stats, stats, x, weight_dtype=torch.bfloat16)),
            (TypeError, lambda: qopt.LayerNorm(8, device="cpu", dtype=torch.float16)),
            (ValueError, lambda: qopt.LayerNorm(8, eps=-1.0, device="cpu"))):
        with pytest.raises(err):
            call()


def test_module_parameters():
    m = qopt.LayerNorm(8, device="cpu", dtype=torch.bfloat16)
    assert sorted(m.state_dict()) == ["bias", "weight"] and m.weight.dtype == torch.bfloat16
    assert torch.equal(m.weight.float(), torch.ones(8)) and not m.bias.any()
    assert sorted(qopt.LayerNorm(8, bias=False, device="cpu").state_dict()) == ["weight"]
