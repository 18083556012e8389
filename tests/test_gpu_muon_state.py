"""GPU tests of the Muon optimizer's state: refused steps leave none, and what is loaded can be stepped."""

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import block_wise_bit_adam8bit_amd as q
    torch.cuda.set_device(0)
    return q


def params(seed, shapes=((96, 64), (40, 96), (64, 64), (8, 16))):
    rng = np.random.default_rng(seed)
    ps = [torch.nn.Parameter(torch.from_numpy((rng.normal(size=s) * 0.02).astype(np.float32)).cuda()) for s in shapes]
    for p in ps:
        p.grad = torch.from_numpy((rng.normal(size=p.shape) * 1e-3).astype(np.float32)).cuda()
    return ps


def test_a_refused_step_leaves_no_entries(q, monkeypatch):
    ps = params(0)
    opt = q.Muon([dict(params=ps[:2]), dict(params=ps[2:])], min_8bit_size=1)

    def refused(error):
        with pytest.raises(error):
            opt.step()
        assert not opt.state and not opt.state_dict()["state"]

    opt.param_groups[1]["lr"] = -1.0
    refused(q.QoptError)
    opt.param_groups[1]["lr"] = 1e-3
    ps[3].grad = ps[3].grad.t().contiguous().t()
    refused(RuntimeError)
    ps[3].grad = ps[3].grad.contiguous()
    with monkeypatch.context() as m:
        m.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
        refused(RuntimeError)
    other = q.Muon([dict(params=ps[:2]), dict(params=ps[2:])])
    other.load_state_dict(opt.state_dict())
    opt.step()
    assert all(opt.state[p] for p in ps)


def test_the_codebook_comes_with_coded_state(q, monkeypatch):
    """A process that loads its state may capture its first step: the codebook, whose first copy cannot be captured,
    is on the device by then.  So it is after the state's conversion and after a first step."""
    from block_wise_bit_adam8bit_amd import functional, muon
    ps = params(1)
    first = q.Muon(ps, min_8bit_size=1)
    first.step()
    saved = first.state_dict()
    for p in ps:
        p.grad = torch.ones_like(p) * 1e-3
    before = [p.detach().clone() for p in ps]
    cache = {}
    monkeypatch.setattr(functional, "_cb_cache", cache)
    opt = q.Muon(ps, min_8bit_size=1)
    opt.load_state_dict(saved)
    assert (muon.SIGNED, 0) in cache
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        opt.step()
    assert all(torch.equal(p, b) for p, b in zip(ps, before))
    twin = [torch.nn.Parameter(p.detach().clone()) for p in ps]
    other = q.Muon(twin, min_8bit_size=1)
    other.load_state_dict(saved)
    for t, p in zip(twin, ps):
        t.grad = p.grad.clone()
    for _ in range(3):
        graph.replay()
        other.step()
        torch.cuda.synchronize()
        assert all(torch.equal(p, t) for p, t in zip(ps, twin))
    cache.clear()
    opt = q.Muon([torch.nn.Parameter(torch.ones(64, 64, device="cuda"))])
    p, = opt.param_groups[0]["params"]
    p.grad = torch.ones_like(p)
    opt._init_states(opt.param_groups[0], [p])
    assert (muon.SIGNED, 0) in cache
