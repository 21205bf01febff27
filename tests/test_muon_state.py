"""The Muon optimiser's state and groups, without a GPU: the orthogonalisation
is replaced by a plain one."""
import copy
import io

import pytest
import torch

from differentiable_gaussian_splatting_pdr_amd import dense


@pytest.fixture(autouse=True)
def plain(monkeypatch):
    monkeypatch.setattr(dense, "orthogonalize", lambda g, *a, dtype=None, **k: (
        g.double() / g.double().norm(dim=(-2, -1), keepdim=True)).to(dtype or g.dtype))


def weights(dtype):
    gen = torch.Generator().manual_seed(1)
    return [torch.randn(*s, generator=gen).to(dtype).requires_grad_() for s in ((8, 6), (8, 6), (5, 9))]


def walk(opt, ps, start, stop):
    for k in range(start, stop):
        gen = torch.Generator().manual_seed(100 + k)
        for p in ps:
            p.grad = (torch.randn(*p.shape, generator=gen) * 0.01).to(p.dtype)
        opt.step()


@pytest.mark.parametrize("state", [torch.float32, torch.bfloat16, torch.float64])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_a_reloaded_optimiser_goes_on_as_the_other_would_have(dtype, state):
    ps = weights(dtype)
    opt = dense.Muon(ps, lr=0.1, state_dtype=state)
    walk(opt, ps, 0, 3)
    file = io.BytesIO()
    torch.save({"opt": opt.state_dict(), "ps": [p.detach() for p in ps]}, file)
    file.seek(0)
    saved = torch.load(file, weights_only=True)
    # with other arguments: the groups' own are loaded
    qs = [p.clone().requires_grad_() for p in saved["ps"]]
    other = dense.Muon(qs, lr=0.5, state_dtype=torch.float32)
    other.load_state_dict(saved["opt"])
    for p, q in zip(ps, qs):
        a, b = opt.state[p]["momentum"], other.state[q]["momentum"]
        assert b.dtype == state and torch.equal(a, b)
    walk(opt, ps, 3, 6)
    walk(other, qs, 3, 6)
    for p, q in zip(ps, qs):
        assert torch.equal(p, q)


def test_loading_shares_nothing_and_runs_the_hooks():
    ps = weights(torch.bfloat16)
    opt = dense.Muon(ps)
    walk(opt, ps, 0, 2)
    qs = [p.detach().clone().requires_grad_() for p in ps]
    other, seen = dense.Muon(qs), []

    def halve(_, given):
        given = copy.deepcopy(given)
        for s in given["state"].values():
            s["momentum"] *= 0.5
        return given
    other.register_load_state_dict_pre_hook(halve)
    other.register_load_state_dict_post_hook(lambda o: seen.append(o.state[qs[0]]["momentum"].dtype))
    other.load_state_dict(opt.state_dict())
    before = opt.state[ps[0]]["momentum"].clone()
    assert torch.equal(other.state[qs[0]]["momentum"], 0.5 * before) and seen == [torch.float32]
    third = dense.Muon(qs)
    third.load_state_dict(opt.state_dict())
    walk(third, qs, 2, 3)
    assert torch.equal(opt.state[ps[0]]["momentum"], before)
    # a copy of the optimiser loads too
    again = copy.deepcopy(opt)
    again.load_state_dict(opt.state_dict())
    # a weight that has had no gradient has no state
    fresh = dense.Muon(weights(torch.bfloat16))
    dense.Muon(weights(torch.bfloat16)).load_state_dict(fresh.state_dict())


def test_every_group_is_checked():
    w = torch.zeros(4, 3, requires_grad=True)
    for shape in ((3,), (2, 3, 4), (2, 3, 4, 5), ()):
        bad = torch.zeros(shape, requires_grad=True)
        with pytest.raises(ValueError):
            dense.Muon([w, bad])
        opt = dense.Muon([w])
        with pytest.raises(ValueError):
            opt.add_param_group({"params": [torch.zeros(2, 2, requires_grad=True), bad]})
        assert len(opt.param_groups) == 1
    for kw in (dict(lr=-1.0), dict(momentum=1.0), dict(momentum=-0.1), dict(weight_decay=-1.0), dict(steps=-1),
               dict(steps=1.5), dict(coefficients=(1.0, 2.0)), dict(work_dtype=torch.float64), dict(state_dtype=torch.int32)):
        with pytest.raises(ValueError):
            dense.Muon([w], **kw)
        with pytest.raises(ValueError):
            dense.Muon([{"params": [w], **kw}])
        opt = dense.Muon([w])
        with pytest.raises(ValueError):
            opt.add_param_group({"params": [torch.zeros(2, 2, requires_grad=True)], **kw})
        assert len(opt.param_groups) == 1
    opt.add_param_group({"params": torch.zeros(2, 2, requires_grad=True), "lr": 0.5})
    assert opt.param_groups[1]["lr"] == 0.5 and opt.param_groups[1]["steps"] == 5
