"""GPU tests that a refused AdamW step leaves everything as it was: parameters of every group,
states and step counts."""

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import block_wise_bit_adam8bit_amd as q
    torch.cuda.set_device(0)
    return q


def groups(q, second, **options):
    """An optimizer of one ordinary group and ``second``, each parameter 1 with gradient 1."""
    first = [torch.nn.Parameter(torch.ones(64, 64, device="cuda")), torch.nn.Parameter(torch.ones(9, device="cuda"))]
    for p in [*first, *second]:
        p.data.fill_(1)
        p.grad = torch.ones_like(p)
    return q.AdamW([dict(params=first), dict(params=second, **options)])


def snapshot(opt):
    return [(p.detach().clone(), {k: v.clone() if torch.is_tensor(v) else v for k, v in opt.state[p].items()})
            for g in opt.param_groups for p in g["params"]]


def same(a, b):
    return all(torch.equal(p, r) and s.keys() == t.keys() and
               all(torch.equal(s[k], t[k]) if torch.is_tensor(s[k]) else s[k] == t[k] for k in s)
               for (p, s), (r, t) in zip(a, b))


@pytest.mark.parametrize("bits", [8, 32])
def test_overlapping_parameters(q, bits):
    room = torch.empty(10000, device="cuda")
    opt = groups(q, [torch.nn.Parameter(room[:6000]), torch.nn.Parameter(room[4000:])], state_bits=bits)
    before = snapshot(opt)
    with pytest.raises(ValueError, match="overlap"):
        opt.step()
    assert same(snapshot(opt), before) and not any(opt.state.values())


@pytest.mark.parametrize("started", [False, True])
@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("change", [dict(lr=float("nan")), dict(lr=float("inf")), dict(eps=-1.0),
                                    dict(betas=(0.9, 1.0)), dict(weight_decay=-0.5)])
def test_settings_of_a_later_group(q, change, bits, started):
    opt = groups(q, [torch.nn.Parameter(torch.empty(5000, device="cuda"))], state_bits=bits)
    if started:
        opt.step()
    before = snapshot(opt)
    good = dict(opt.param_groups[1])
    opt.param_groups[1].update(change)
    with pytest.raises((ValueError, q.QoptError)):
        opt.step()
    assert same(snapshot(opt), before) and any(opt.state.values()) == started
    opt.param_groups[1].update(good)
    opt.step()
    assert all(opt.state[p]["step"] == 1 + started for g in opt.param_groups for p in g["params"])


@pytest.mark.parametrize("scale", [(torch.ones, 2), (torch.ones, 0), (torch.zeros, (1, 1), torch.float64)])
def test_grad_scale(q, scale):
    opt = groups(q, [torch.nn.Parameter(torch.empty(5000, device="cuda"))])
    make, shape, *dtype = scale
    with pytest.raises(ValueError, match="one float32 value"):
        opt.step(grad_scale=make(shape, device="cuda", dtype=dtype[0] if dtype else None))
    assert not any(opt.state.values())
    assert all(bool((p == 1).all()) for g in opt.param_groups for p in g["params"])
