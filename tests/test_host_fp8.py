"""CPU tests of the 8-bit product entry points' argument checks: nothing reaches the
device."""

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
    assert c["QOPT_FP8_BLOCK"] == _lib.QOPT_FP8_BLOCK == 128
    assert c["QOPT_FP8_MAX_DIM"] == _lib.QOPT_FP8_MAX_DIM
    assert c["QOPT_FP8_FEW_ROWS"] == _lib.QOPT_FP8_FEW_ROWS


def test_quantize_checks():
    def call(x=P, dt=0, rows=4, cols=256, ldx=256, form=0, c=P, s=P, ct=P, st=P):
        return L.qopt_fp8_quantize(x, dt, rows, cols, ldx, form, c, s, ct, st, None)

    assert call(rows=0) == OK and call(cols=0, ldx=0, x=None) == OK
    for bad in (dict(rows=-1), dict(cols=-1), dict(rows=_lib.QOPT_FP8_MAX_DIM + 1), dict(ldx=255),
                dict(cols=_lib.QOPT_FP8_MAX_DIM + 1, ldx=1 << 40), dict(x=None), dict(c=None),
                dict(s=None), dict(ct=None), dict(st=None), dict(c=None, s=None, ct=None, st=None),
                dict(rows=1 << 23, cols=1 << 23, ldx=1 << 23)):
        assert call(**bad) == EINVAL, bad
    for bad in (dict(dt=2), dict(dt=-1), dict(form=2), dict(form=-1)):
        assert call(**bad) == EUNSUPPORTED, bad
    for bad in (dict(x=P + 2), dict(x=P + 1, dt=1), dict(c=P + 8), dict(ct=P + 8)):
        assert call(**bad) == EALIGN, bad


def test_matmul_checks():
    def call(a=P, sa=P, b=P, sb=P, fb=0, m=4, n=8, k=256, out=P, dt=1, ldo=8, ws=None, nws=0):
        return L.qopt_fp8_matmul(a, sa, b, sb, fb, m, n, k, out, dt, ldo, ws, nws, None)

    assert call(m=0) == OK and call(n=0, ldo=0, out=None) == OK
    for bad in (dict(m=-1), dict(n=-1), dict(k=-1), dict(ldo=7), dict(a=None), dict(sa=None),
                dict(b=None), dict(sb=None), dict(out=None), dict(k=_lib.QOPT_FP8_MAX_DIM + 1)):
        assert call(**bad) == EINVAL, bad
    for bad in (dict(dt=2), dict(fb=2), dict(fb=-1)):
        assert call(**bad) == EUNSUPPORTED, bad
    for bad in (dict(a=P + 8), dict(b=P + 4), dict(out=P + 1), dict(out=P + 2, dt=0), dict(ws=P + 8),
                dict(sa=P + 2), dict(sb=P + 1)):
        assert call(**bad) == EALIGN, bad


def test_linear_checks():
    def call(x=P, dt=1, m=4, k=256, ldx=256, w=P, sw=P, f=1, n=8, out=P, odt=1, ldo=8, ws=None, nws=0):
        return L.qopt_fp8_linear(x, dt, m, k, ldx, w, sw, f, n, out, odt, ldo, ws, nws, None)

    assert call(m=0) == OK and call(n=0, ldo=0) == OK
    for bad in (dict(m=-1), dict(n=-1), dict(k=-1), dict(ldx=255), dict(ldo=7), dict(x=None),
                dict(w=None), dict(sw=None), dict(out=None), dict(m=33), dict(m=33, ws=P, nws=16)):
        assert call(**bad) == EINVAL, bad
    for bad in (dict(dt=3), dict(odt=3), dict(f=2)):
        assert call(**bad) == EUNSUPPORTED, bad
    for bad in (dict(x=P + 1), dict(x=P + 2, dt=0), dict(w=P + 8), dict(sw=P + 2), dict(out=P + 1),
                dict(m=33, ws=P + 8, nws=1 << 30)):
        assert call(**bad) == EALIGN, bad


def test_workspace_queries():
    n = ctypes.c_size_t(7)
    for q in (L.qopt_fp8_matmul_workspace, L.qopt_fp8_linear_workspace):
        assert q(0, 0, 0, 1, ctypes.byref(n)) == OK and n.value == 0
        assert q(4, 4, 4, 1, None) == EINVAL
        assert q(-1, 4, 4, 1, ctypes.byref(n)) == EINVAL
        assert q(4, 4, _lib.QOPT_FP8_MAX_DIM + 1, 1, ctypes.byref(n)) == EINVAL
        assert q(4, 4, 4, 9, ctypes.byref(n)) == EUNSUPPORTED
    assert L.qopt_fp8_linear_workspace(32, 512, 300, 1, ctypes.byref(n)) == OK and n.value == 0
    assert L.qopt_fp8_linear_workspace(33, 512, 300, 1, ctypes.byref(n)) == OK
    assert n.value >= 33 * 384 + 48 * 3
    assert q(1 << 23, 1 << 23, 128, 1, ctypes.byref(n)) == EINVAL  # too many tiles of results


def test_wrappers_refuse_what_is_not_a_matrix_on_a_gpu():
    x = torch.zeros(4, 256)
    codes = torch.zeros(8, 256, dtype=torch.float8_e4m3fn)
    scales = torch.zeros(1, 2, dtype=torch.uint8)
    for call in (lambda: qopt.qopt_fp8_quantize(x), lambda: qopt.qopt_fp8_linear(x, codes, scales),
                 lambda: qopt.qopt_fp8_matmul(codes, scales, codes, scales),
                 lambda: qopt.fp8_linear(x, torch.zeros(8, 256))):
        with pytest.raises(ValueError):  # on the CPU
            call()
    for err, call in (
            (ValueError, lambda: qopt.qopt_fp8_quantize(x[0])),
            (ValueError, lambda: qopt.qopt_fp8_quantize(x, normal=False)),
            (TypeError, lambda: qopt.qopt_fp8_quantize(x.half())),
            (TypeError, lambda: qopt.qopt_fp8_linear(x.half(), codes, scales)),
            (TypeError, lambda: qopt.qopt_fp8_linear(x, codes.view(torch.uint8), scales)),
            (TypeError, lambda: qopt.qopt_fp8_linear(x, codes, scales.int())),
            (TypeError, lambda: qopt.qopt_fp8_linear(x, codes, scales, torch.float16)),
            (ValueError, lambda: qopt.qopt_fp8_linear(x, codes[:, :200], scales)),
            (ValueError, lambda: qopt.qopt_fp8_linear(x, codes, scales.repeat(2, 1))),
            (ValueError, lambda: qopt.qopt_fp8_linear(x, codes, scales[:, :1])),
            (ValueError, lambda: qopt.qopt_fp8_linear(x[:, :128], codes, scales)),
            (ValueError, lambda: qopt.qopt_fp8_linear(x.t().contiguous().t(), codes, scales)),
            (ValueError, lambda: qopt.qopt_fp8_linear(x[:1].expand(4, 256), codes, scales)),
            (ValueError, lambda: qopt.qopt_fp8_matmul(codes, scales, codes[:, :128].contiguous(),
                                                      scales[:, :1].contiguous())),
            (TypeError, lambda: qopt.fp8_linear(x, torch.zeros(8, 256).half())),
            (ValueError, lambda: qopt.fp8_linear(x, torch.zeros(8, 255)))):
        with pytest.raises(err):
            call()
