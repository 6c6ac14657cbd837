"""Offsets that decrease or leave the token rows: a new result holds zeros, never what its memory held
before, and the gradients that autograd hands on are zero too (needs a B200)."""
import pytest

pytestmark = pytest.mark.gpu

# (token rows, rows N, columns K, experts): few tokens (fp32: split by the kernel), many (fp32: packed), CTA pairs
SIZES = {"few": (40, 72, 64, 3), "odd": (41, 77, 65, 3), "many": (400, 136, 88, 3), "paired": (4200, 1536, 96, 4)}
BAD = {"decreasing": lambda t: [0, t // 2, t // 3, t], "too_far": lambda t: [0, 5, 9, t + 1], "negative": lambda t: [-1, 5, 9, t],
       "large": lambda t: [2147483647, 0, 1, 2]}


@pytest.fixture(scope="module")
def muon():
    from spectral_optimizer_state_b200 import Muon
    with Muon(0) as mu:
        yield mu


def _offsets(bad, tokens, experts):
    import torch
    o = BAD[bad](tokens)
    return torch.tensor(o + [o[-1]] * (experts + 1 - len(o)), dtype=torch.int32, device="cuda")


def _stain(*shapes, dtype):
    """Leaves NaN in the blocks that the next allocations of these shapes take."""
    import torch
    kept = [torch.full(s, float("nan"), dtype=dtype, device="cuda") for s in shapes for _ in range(3)]
    torch.cuda.synchronize()
    del kept


def _reported(muon):
    from spectral_optimizer_state_b200 import MuonError
    with pytest.raises(MuonError) as err:
        muon.status()
    return err.value.status == 1


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("size", list(SIZES))
@pytest.mark.parametrize("bad", list(BAD))
def test_new_results_and_gradients_are_zero(muon, bad, size, dtype):
    import torch
    from spectral_optimizer_state_b200 import expert_linear
    tokens, n, k, experts = SIZES[size]
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    off = _offsets(bad, tokens, experts)
    x = torch.ones(tokens, k, dtype=dt, device="cuda").requires_grad_()
    w = torch.ones(experts, n, k, dtype=dt, device="cuda").requires_grad_()
    dy = torch.ones(tokens, n, dtype=dt, device="cuda")
    _stain((tokens, n), (tokens, k), (experts, n, k), dtype=dt)
    y = muon.expert_matmul(x.detach(), w.detach(), off)
    dx = muon.expert_matmul(dy, w.detach(), off, transpose=True)
    assert not y.any() and not dx.any()
    del y, dx
    _stain((tokens, n), (tokens, k), (experts, n, k), dtype=dt)
    h = expert_linear(x, w, off, muon)
    h.backward(dy)
    assert not h.any() and not x.grad.any() and not w.grad.any()
    assert _reported(muon)


@pytest.mark.parametrize("size", list(SIZES))
def test_the_callers_buffers_are_left_alone(muon, size):
    """With out given nothing is written, neither the rows nor a gradient that is overwritten or added to."""
    import torch
    tokens, n, k, experts = SIZES[size]
    for dt in (torch.bfloat16, torch.float32):
        off = _offsets("decreasing", tokens, experts)
        x, w = torch.ones(tokens, k, dtype=dt, device="cuda"), torch.ones(experts, n, k, dtype=dt, device="cuda")
        dy, y = torch.ones(tokens, n, dtype=dt, device="cuda"), torch.full((tokens, n), 7.0, dtype=dt, device="cuda")
        muon.expert_matmul(x, w, off, out=y)
        assert bool((y == 7.0).all())
        for out in {dt, torch.float32}:
            for beta in (0.0, 1.0, 0.5):
                G = torch.full((experts, n, k), 7.0, dtype=out, device="cuda")
                muon.expert_grad(dy, x, off, G, beta=beta)
                assert bool((G == 7.0).all())
        main = torch.full((experts, n, k), 7.0, device="cuda")
        wr = w.clone().requires_grad_()
        from spectral_optimizer_state_b200 import expert_linear
        expert_linear(x, wr, off, muon, grad_into=main).sum().backward()
        assert bool((main == 7.0).all())
        assert _reported(muon)


def test_good_offsets_write_every_element_of_a_new_gradient(muon):
    """The gradient of a new result, as autograd gets it: every element written, experts without rows zero, and
    equal to the gradient that overwrites a buffer of the caller's."""
    import torch
    from spectral_optimizer_state_b200 import expert_linear
    for dt in (torch.bfloat16, torch.float32):
        for n, k, counts in ((77, 65, [3, 0, 40]), (136, 88, [200, 0, 250]), (1, 1, [0, 0, 0])):
            o = [0]
            for c in counts:
                o.append(o[-1] + c)
            off = torch.tensor(o, dtype=torch.int32, device="cuda")
            x = torch.randn(o[-1], k, device="cuda").to(dt)
            w = torch.randn(3, n, k, device="cuda").to(dt).requires_grad_()
            dy = torch.randn(o[-1], n, device="cuda").to(dt)
            want = muon.expert_grad(dy, x, off, torch.full((3, n, k), 7.0, dtype=dt, device="cuda"), beta=0.0)
            _stain((3, n, k), dtype=dt)
            expert_linear(x, w, off, muon).backward(dy)
            assert torch.equal(w.grad, want) and not w.grad[1].any()
    assert muon.status()[0] == 0


def test_a_new_gradient_takes_no_beta(muon):
    import torch
    from spectral_optimizer_state_b200 import MuonError
    off = torch.tensor([0, 4], dtype=torch.int32, device="cuda")
    x, dy = torch.ones(4, 8, device="cuda"), torch.ones(4, 6, device="cuda")
    with pytest.raises(ValueError):
        muon.expert_grad(dy, x, off, beta=1.0)
    with pytest.raises(MuonError):
        muon.expert_grad(dy, x, off[:1])  # no experts
    G = muon.expert_grad(dy, x, off, scale=0.5)
    assert G.shape == (1, 6, 8) and G.dtype is x.dtype and bool((G == 2.0).all())
