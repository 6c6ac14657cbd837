"""Gradients that are accumulated outside .grad, and gradients of another type than the weights', reach the step."""
import pytest
import torch

from spectral_optimizer_state_b200 import optim


class _Ctx:
    """Keeps what the step would hand to the kernels."""

    def __init__(self, *a, **k):
        self.seen = []

    def step_groups(self, groups, stream=None, **hp):
        self.seen += [(w, g) for W, G, M in groups for w, g in zip(W, G)]

    def step_blocks(self, W, G, M, block, stream=None, **hp):
        self.seen += list(zip(W, G))


@pytest.fixture()
def adam(monkeypatch):
    seen = []
    monkeypatch.setattr(optim, "Muon", _Ctx)
    monkeypatch.setattr(optim, "adamw_step", lambda W, G, *a, **k: seen.extend(zip(W, G)))
    return seen


def _params(dtype):
    return {n: torch.zeros(s, dtype=dtype, requires_grad=True)
            for n, s in (("moe.in_proj", (3, 6, 4)), ("heads.in_proj", (6, 4)), ("whole.in_proj", (6, 4)), ("norm", (4,)))}


def test_fp32_gradients_of_bf16_weights_are_rounded(adam):
    p = _params(torch.bfloat16)
    opt = optim.MuonAdamW(list(p.items()), stacked=True, blocks={"heads": (3, None)})
    grads = {n: torch.full(t.shape, 1.0 + 2.0 ** -12) for n, t in p.items()}
    kept = {n: g.clone() for n, g in grads.items()}
    opt.step(grads)
    for w, g in opt.ctx.seen + adam:
        assert g.dtype is w.dtype is torch.bfloat16 and g.shape == w.shape and bool((g == 1.0).all())
    assert len(opt.ctx.seen) == 5 and len(adam) == 1
    assert all(torch.equal(grads[n], kept[n]) for n in grads)  # the buffers keep their bits


def test_gradients_of_the_weights_type_are_taken_as_they_are(adam):
    p = _params(torch.float32)
    opt = optim.MuonAdamW(list(p.items()), stacked=True)
    grads = {n: torch.ones_like(t) for n, t in p.items()}
    opt.step(grads)
    assert [g.data_ptr() for _, g in opt.ctx.seen[:3]] == [m.data_ptr() for m in grads["moe.in_proj"]]
    assert adam[0][1].data_ptr() == grads["norm"].data_ptr()


def test_accumulation_buffers_stand_in_for_grad(adam):
    p = _params(torch.bfloat16)
    main = torch.full((3, 6, 4), 2.0)
    opt = optim.torch_optimizer(list(p.items()), stacked=True, main_grads={"moe.in_proj": main})
    p["whole.in_proj"].grad = torch.ones(6, 4, dtype=torch.bfloat16)
    opt.step()
    ctx = opt.inner.ctx
    assert len(ctx.seen) == 4 and not adam  # the stack's three matrices and the one with a .grad
    assert all(bool((g == 2.0).all()) and g.dtype is torch.bfloat16 for _, g in ctx.seen[:3])
    opt.zero_grad()
    assert not main.any() and p["whole.in_proj"].grad is None
    p["moe.in_proj"].grad = torch.ones(3, 6, 4, dtype=torch.bfloat16)
    with pytest.raises(ValueError):  # which of the two is meant is not known
        opt.step()


@pytest.mark.parametrize("main", [{"moe.out_proj": (3, 6, 4)}, {"moe.in_proj": (3, 4, 6)}])
def test_buffers_of_no_parameter_are_refused(adam, main):
    with pytest.raises(ValueError):
        optim.torch_optimizer(list(_params(torch.bfloat16).items()), stacked=True,
                              main_grads={n: torch.zeros(s) for n, s in main.items()})
