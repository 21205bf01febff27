"""The dense operators' Python side without a GPU: what it passes on, copies
and refuses, with the launches left out."""
import pytest
import torch
from torch.autograd import forward_ad

from differentiable_gaussian_splatting_pdr_amd import dense


@pytest.fixture
def no_launch(monkeypatch):
    """Operators on CPU tensors that launch nothing; the names of the calls they would make."""
    calls = []
    monkeypatch.setattr(dense, "_check", lambda *a: None)
    monkeypatch.setattr(dense, "_call", lambda name, *a: calls.append(name))
    return calls


def operators(x, w_in, w_out, g):
    return ((lambda v: dense.linear(v, w_in), x), (lambda v: dense.linear(x, v, activation="gelu"), w_in),
            (lambda v: dense.linear(x, w_in, residual=v), torch.zeros(5, 12)),
            (lambda v: dense.linear(x, w_in, bias=v), torch.zeros(12)),
            (lambda v: dense.gated_mlp(v, w_in, w_out), x), (lambda v: dense.gated_mlp(x, v, w_out), w_in),
            (lambda v: dense.gated_mlp(x, w_in, w_out, residual=v), torch.zeros(5, 8)), (dense.orthogonalize, g))


def test_forward_mode_is_refused(no_launch):
    # no tangent may be lost without a word
    for f, at in operators(torch.ones(5, 8), torch.ones(12, 8), torch.ones(8, 6), torch.ones(4, 6)):
        for no_grad in (False, True):
            with forward_ad.dual_level(), torch.set_grad_enabled(not no_grad):
                with pytest.raises(NotImplementedError):
                    f(forward_ad.make_dual(at, torch.ones_like(at)))
                f(at)   # nothing is differentiated
        with pytest.raises(RuntimeError):
            torch.func.jvp(f, (at,), (torch.ones_like(at),))
        with pytest.raises(RuntimeError):
            torch.vmap(f)(torch.stack((at, at)))


@pytest.mark.parametrize("apart", [(1 << 22) - 1, 1 << 22, (1 << 22) + 1, 3 << 22])
def test_rows_further_apart_than_the_kernels_take_are_copied(apart, monkeypatch):
    v = torch.arange(2 * apart, dtype=torch.float16).view(2, apart)[:, 5:15]
    rows = dense._rows(v)
    assert torch.equal(rows, v) and dense._ld(rows) == (10 if apart > 1 << 22 else apart)
    # the last token of each sequence
    last = torch.zeros(2, 3, apart // 3 + 1, dtype=torch.float16)[:, -1, :8]
    assert dense._ld(dense._rows(last)) == (8 if 3 * (apart // 3 + 1) > 1 << 22 else 3 * (apart // 3 + 1))
    seen = []
    monkeypatch.setattr(dense, "_check", lambda *a: None)
    monkeypatch.setattr(dense, "_call", lambda name, args, device: seen.append((args.ldg, args.batch_g)))
    dense.orthogonalize(v)
    dense.orthogonalize(torch.stack((v, v))[:1])
    assert seen == [(10 if apart > 1 << 22 else apart, 0), (10, 20)]


@pytest.mark.parametrize("shape", [(2, 0, 8), (0, 3, 8), (2, 3, 0), (0,)])
def test_inputs_without_elements_keep_their_gradient(no_launch, shape):
    x, n = torch.zeros(*shape, requires_grad=True), shape[-1]
    for y in (dense.linear(x, torch.ones(4, n)), dense.gated_mlp(x, torch.ones(6, n), torch.ones(4, 3))):
        assert y.shape == (*shape[:-1], 4) and y.requires_grad
        (g,) = torch.autograd.grad(y.sum(), x)
        assert g.shape == x.shape
    r = torch.zeros(*shape[:-1], 4, requires_grad=True)
    y = dense.linear(x.detach(), torch.ones(4, n), residual=r)
    assert y.requires_grad and torch.autograd.grad(y.sum(), r)[0].shape == r.shape


def test_kept_rows_are_as_far_apart_as_the_library_says():
    from differentiable_gaussian_splatting_pdr_amd import _lib
    for n in (0, 1, 7, 8, 9, 1000, 1 << 22):
        assert dense._kept_ld(n) == _lib.pdr_dense_kept_ld(n)
