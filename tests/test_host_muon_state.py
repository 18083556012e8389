"""CPU tests of what the Muon optimizer's loader takes and refuses."""

import pytest
import torch

qopt = pytest.importorskip("block_wise_bit_adam8bit_amd")


def optimizer(*shapes):
    return qopt.Muon([torch.nn.Parameter(torch.zeros(s)) for s in shapes])


def test_a_parameter_without_state_is_loaded_as_one():
    """An entry without anything in it, as a dict that is asked for a missing parameter's state makes it."""
    opt = optimizer((4, 4), (3, 5))
    saved = opt.state_dict()
    saved["state"] = {0: {}, 1: dict(momentum_buffer=torch.ones(3, 5))}
    opt.load_state_dict(saved)
    a, b = opt.param_groups[0]["params"]
    assert a not in opt.state and torch.equal(opt.state[b]["momentum_buffer"], torch.ones(3, 5))


def test_a_parameter_without_state_converts_to_none():
    opt = optimizer((4, 4), (3, 5))
    opt.state[opt.param_groups[0]["params"][0]]  # a look at it makes an entry
    if hasattr(torch.optim, "Muon"):
        assert not opt.fp32_muon_state_dict()["state"]
    saved = opt.state_dict()
    for g in saved["param_groups"]:
        g["adjust_lr_fn"] = g["adjust"]
    saved["state"] = {0: {}, 1: {}}
    opt.load_fp32_muon_state(saved)
    assert not opt.state


def test_a_codebook_is_not_copied_inside_of_a_capture(monkeypatch):
    from block_wise_bit_adam8bit_amd import functional
    monkeypatch.setattr(functional, "_cb_cache", {})
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
    with pytest.raises(RuntimeError, match="captured"):
        functional.codebook(functional.SIGNED, torch.device("cuda", 0))
    assert not functional._cb_cache


def test_momentum_of_another_shape_is_refused():
    opt = optimizer((3, 5))
    p, = opt.param_groups[0]["params"]
    saved = opt.state_dict()
    for shape in ((5, 3), (15,), (1, 15)):  # as many elements as the parameter has
        saved["state"] = {0: dict(momentum_buffer=torch.ones(shape))}
        with pytest.raises(ValueError, match="shape"):
            opt.load_state_dict(saved)
        assert not opt.state
    m = torch.arange(15.0).view(5, 3).t()  # its shape, in another order of memory
    saved["state"] = {0: dict(momentum_buffer=m)}
    opt.load_state_dict(saved)
    assert torch.equal(opt.state[p]["momentum_buffer"], m) and opt.state[p]["momentum_buffer"].is_contiguous()
