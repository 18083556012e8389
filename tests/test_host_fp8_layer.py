"""CPU tests of the 8-bit linear layer's Python side: what reaches the library and what torch
records of it.  The library's calls are replaced by a stand-in that fills the results."""

import ctypes

import numpy as np
import pytest
import torch

qopt = pytest.importorskip("block_wise_bit_adam8bit_amd")
from block_wise_bit_adam8bit_amd import _lib, fp8  # noqa: E402

VALUE = 7.0


@pytest.fixture
def calls(monkeypatch):
    """Names of the library's entry points as they are called; results are float32 VALUEs.
    Arguments have to be such as ctypes takes for the entry point."""
    names = []

    def call(name, device, *args):
        names.append(name)
        for kind, arg in zip(_lib._SIGNATURES[name][1], (*args, None), strict=True):
            kind.from_param(arg) if kind is ctypes.c_void_p else kind(arg)
        if name == "qopt_fp8_matmul":
            out, m, n, ldo = args[8], args[5], args[6], args[10]
        elif name == "qopt_fp8_linear":
            out, m, n, ldo = args[9], args[2], args[8], args[11]
        else:
            return
        for row in range(m):
            np.ctypeslib.as_array((ctypes.c_float * n).from_address(out + 4 * row * ldo))[:] = VALUE

    monkeypatch.setattr(_lib, "call", call)
    monkeypatch.setattr(fp8, "_same_gpu", lambda first, *others: first.device)
    return names


class Layer(torch.nn.Module):
    def __init__(self, requires_grad):
        super().__init__()
        self.weight = torch.nn.Parameter(torch.randn(24, 200), requires_grad=requires_grad)

    def forward(self, x):
        return qopt.fp8_linear(x, self.weight)


@pytest.mark.parametrize("m", [3, 40])
@pytest.mark.parametrize("requires_grad", [False, True])
@pytest.mark.parametrize("grad_mode", [False, True])
def test_a_traced_layer_calls_the_library(calls, grad_mode, requires_grad, m):
    """A trace holds the products themselves, whatever gradients were wanted while it was made."""
    layer = Layer(requires_grad)
    with torch.set_grad_enabled(grad_mode):
        traced = torch.jit.trace(layer, (torch.randn(m, 200),))
        del calls[:]
        y = traced(torch.randn(m, 200))
    assert calls and calls[-1] in ("qopt_fp8_linear", "qopt_fp8_matmul")
    assert y.shape == (m, 24) and bool((y == VALUE).all())
    # gradients are those of the mode it runs in, not of the one it was traced in
    y = traced(torch.randn(m + 30, 200))
    assert y.shape == (m + 30, 24)
    assert y.requires_grad == requires_grad and bool((y == VALUE).all())
    if requires_grad:
        assert torch.autograd.grad(y.sum(), list(traced.parameters()))[0].shape == (24, 200)


def test_a_backward_pass_is_not_traced(calls):
    """Its gradients would be empty tensors in a trace: refused, instead of wrong."""
    w = torch.randn(24, 200)
    f = lambda a: torch.autograd.grad(qopt.fp8_linear(a, w).sum(), a)[0]  # noqa: E731
    x = torch.randn(5, 200, requires_grad=True)
    f(x)
    with pytest.raises(RuntimeError, match="trace"):
        torch.jit.trace(f, (x,))


@pytest.mark.parametrize("requires_grad", [False, True])
@pytest.mark.parametrize("grad_mode", [False, True])
@pytest.mark.parametrize("which", ["x", "w"])
def test_forward_mode_is_refused(calls, which, grad_mode, requires_grad):
    """A tangent is not dropped, whether or not gradients are wanted beside it."""
    x, w = torch.randn(5, 200), torch.randn(24, 200)
    with torch.autograd.forward_ad.dual_level(), torch.set_grad_enabled(grad_mode):
        t = x if which == "x" else w
        dual = torch.autograd.forward_ad.make_dual(t, torch.ones_like(t))
        x, w = (dual, w.requires_grad_(requires_grad)) if which == "x" else (x.requires_grad_(requires_grad), dual)
        with pytest.raises(NotImplementedError):
            qopt.fp8_linear(x, w)
        # without a tangent the level itself is no reason to refuse
        assert bool((qopt.fp8_linear(torch.randn(5, 200), torch.randn(24, 200)) == VALUE).all())
    with pytest.raises(RuntimeError):  # functorch's duals hide in wrappers
        torch.func.jvp(lambda a: qopt.fp8_linear(a, torch.randn(24, 200)), (torch.randn(5, 200),), (torch.ones(5, 200),))


def test_the_library_calls_themselves_are_not_traced(calls):
    """Their results would be empty tensors in a trace: refused, instead of wrong."""
    x, codes = torch.randn(5, 256), torch.zeros(24, 256, dtype=torch.uint8).view(torch.float8_e4m3fn)
    tiles, rows = torch.zeros(1, 2, dtype=torch.uint8), torch.zeros(2, 32, dtype=torch.uint8)
    for f in (lambda a: qopt.qopt_fp8_linear(a, codes, tiles),
              lambda a: qopt.qopt_fp8_matmul(codes, rows, codes, tiles, torch.float32) + a.sum(),
              lambda a: qopt.qopt_fp8_quantize(a)[0]):
        f(x)
        with pytest.raises(RuntimeError, match="trace"):
            torch.jit.trace(f, (x,))
    assert len(calls) == 3


def test_layers_start_apart(monkeypatch):
    """Two layers of one shape do not start with the same weights unless they are told to, and
    torch's seed settles which ones they get."""
    seeds = []
    monkeypatch.setattr(fp8, "qopt_embedding_xavier_init", lambda weight, seed: seeds.append(seed))

    def make(**options):
        return qopt.Fp8Linear(16, 16, device="cpu", **options).seed

    torch.manual_seed(5)
    drawn = [make(), make()]
    assert drawn[0] != drawn[1]
    torch.manual_seed(5)
    assert [make(), make()] == drawn
    assert [make(seed=3), make(seed=3), make(seed=0)] == [3, 3, 0]
    assert seeds == [*drawn, *drawn, 3, 3, 0]


def test_out_between_the_rows_of_an_operand(calls):
    """Rows of one buffer side by side do not overlap, whatever their types; rows that share a byte do."""
    codes, tiles = torch.zeros(8, 256, dtype=torch.uint8).view(torch.float8_e4m3fn), torch.zeros(1, 2, dtype=torch.uint8)
    run = lambda x, out: qopt.qopt_fp8_linear(x, codes, tiles, torch.float32, out=out)  # noqa: E731
    for m in (1, 2, 40):
        room = torch.zeros(m, 300)
        for x, out in ((room[:, 8:264], room[:, :8]), (room[:, :256], room[:, 256:264]),
                       (room[:, 30:286], room[:, 22:30]), (room[:, 30:286], room[:, 286:294])):
            run(x, out)
            assert bool((out == VALUE).all()) and bool((x == 0).all())
            room.zero_()
        half = room.view(torch.bfloat16)  # rows of 600
        run(half[:, 17:273], room[:, :8])
        run(half[:, 16:272], room[:, 136:144])
        bad = [(room[:, 7:263], room[:, :8]), (room[:, :256], room[:, 255:263]),
               (room[:, 30:286], room[:, 30:38]), (room[:, 30:286], room[:, 278:286]),
               (half[:, 15:271], room[:, :8]), (half[:, 17:273], room[:, 136:144])]
        if m > 1:  # the next row: columns that run over a row's end, and another distance of the rows
            flat = torch.zeros(m * 300 + 300)
            bad += [(flat.as_strided((m, 256), (300, 1), 100), flat.as_strided((m, 8), (300, 1), 350)),
                    (flat.as_strided((m, 256), (300, 1), 0), flat.as_strided((m, 8), (298, 1), 260))]
        for x, out in bad:
            with pytest.raises(ValueError, match="overlap"):
                run(x, out)
    # an operand that is not rows of a matrix: its whole span counts
    room = torch.zeros(4, 3, 256)
    with pytest.raises(ValueError, match="overlap"):
        run(room, room.view(-1)[:96].view(4, 3, 8))


def test_the_function_itself_checks_its_operands(monkeypatch):
    """As fp8_linear does: a traced layer, too, may be given something else than it was traced with."""
    apply, x, w = qopt.Fp8LinearFunction.apply, torch.randn(5, 200), torch.randn(24, 200)
    with pytest.raises(ValueError, match="on a GPU"):  # before an address on the host goes to the device
        apply(x, w)
    with pytest.raises(ValueError, match="on a GPU"):
        apply(x.requires_grad_(), w)
    monkeypatch.setattr(fp8, "_same_gpu", lambda first, *others: first.device)
    monkeypatch.setattr(_lib, "call", lambda *args: pytest.fail("reached the library"))
    for error, a, b in ((TypeError, x.half(), w), (TypeError, x, w.double()), (ValueError, x, w[:, :199]),
                        (ValueError, x, w.view(-1)), (ValueError, x.sum(), w), (ValueError, x.view(4, 250), w)):
        for f in (apply, qopt.fp8_linear):
            with pytest.raises(error):
                f(a, b)
