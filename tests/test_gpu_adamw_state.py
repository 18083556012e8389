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


def test_a_plan_brings_the_codebooks(q, monkeypatch):
    """A step of a plan may be captured as the first work of a process: the codebooks, whose first copy cannot be
    captured, are on the device by then."""
    from block_wise_bit_adam8bit_amd import functional
    cache = {}
    monkeypatch.setattr(functional, "_cb_cache", cache)
    n = 5000
    state = lambda: (torch.full((n,), 0.5, device="cuda"), torch.full((n,), 0.1, device="cuda"),  # noqa: E731
                     *(torch.zeros(n, dtype=torch.uint8, device="cuda") for _ in range(2)),
                     *(torch.zeros(3, device="cuda") for _ in range(2)))
    a, b = state(), state()
    plan = q.qopt_adamw8bit_plan([a])
    assert {(q.SIGNED, 0), (q.UNSIGNED, 0)} <= set(cache)
    hp = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.1, step=1)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q.qopt_adamw8bit_step(plan, **hp)
    for _ in range(3):
        graph.replay()
        q.qopt_adamw8bit_step([b], **hp)
        torch.cuda.synchronize()
        assert all(torch.equal(s, t) for s, t in zip(a, b))
