"""GPU test of the AdamW optimizer's state: refused steps leave none."""

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import block_wise_bit_adam8bit_amd as q
    torch.cuda.set_device(0)
    return q


def test_a_refused_step_leaves_no_entries(q):
    ps = [torch.nn.Parameter(torch.ones(s, device="cuda")) for s in ((96, 64), (40,), (64, 64), (8, 16))]
    for p in ps:
        p.grad = torch.ones_like(p)
    opt = q.AdamW([dict(params=ps[:2]), dict(params=ps[2:])])

    def refused(error):
        with pytest.raises(error):
            opt.step()
        assert not opt.state and not opt.state_dict()["state"]

    opt.param_groups[1]["weight_decay"] = -1.0
    refused(q.QoptError)
    opt.param_groups[1]["weight_decay"] = 0.0
    ps[3].grad = ps[3].grad.t().contiguous().t()
    refused(RuntimeError)
    ps[3].grad = ps[3].grad.contiguous()
    other = q.AdamW([dict(params=ps[:2]), dict(params=ps[2:])])
    other.load_state_dict(opt.state_dict())
    opt.step()
    assert all(opt.state[p] for p in ps)
