"""CPU tests of what the AdamW optimizer's loader takes."""

import pytest
import torch

qopt = pytest.importorskip("block_wise_bit_adam8bit_amd")


def test_a_parameter_without_state_is_loaded_as_one():
    """An entry without anything in it, as a dict that is asked for a missing parameter's state makes it."""
    a, b = (torch.nn.Parameter(torch.zeros(s)) for s in ((4,), (3, 5)))
    opt = qopt.AdamW([a, b])
    saved = opt.state_dict()
    saved["state"] = {0: {}, 1: dict(step=2, exp_avg=torch.ones(3, 5), exp_avg_sq=torch.ones(3, 5))}
    opt.load_state_dict(saved)
    assert a not in opt.state and opt.state[b]["step"] == 2 and torch.equal(opt.state[b]["exp_avg"], torch.ones(3, 5))
