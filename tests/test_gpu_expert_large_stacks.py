"""Stacks whose elements lie beyond 2^31: weights read and gradients written in the last expert (needs a B200)."""
import pytest

pytestmark = pytest.mark.gpu

U = 2.0 ** -23


@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_the_last_expert_of_a_large_stack(out):
    import torch
    from spectral_optimizer_state_b200 import Muon
    e, n, k = 70, 5640, 5568  # 2.2e9 elements
    assert (e - 1) * n * k > 2 ** 31
    counts = {0: 3, 40: 17, e - 1: 5}
    o = [0]
    for i in range(e):
        o.append(o[-1] + counts.get(i, 0))
    off = torch.tensor(o, dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    x = torch.randn(o[-1], k, generator=g, device="cuda").bfloat16()
    dy = torch.randn(o[-1], n, generator=g, device="cuda").bfloat16()
    with Muon(0) as mu:
        if out == "bf16":
            w = torch.zeros(e, n, k, dtype=torch.bfloat16, device="cuda")
            for i in counts:
                w[i] = 0.05 * torch.randn(n, k, generator=g, device="cuda")
            y, dx = mu.expert_matmul(x, w, off), mu.expert_matmul(dy, w, off, transpose=True)
            for i in counts:
                s = slice(o[i], o[i + 1])
                for got, a, b in ((y[s], x[s].double(), w[i].double().T), (dx[s], dy[s].double(), w[i].double())):
                    ref, mag = a @ b, a.abs() @ b.abs()
                    # additions that truncate, 16 products at a time, and the result's rounding
                    tol = 2 * (a.shape[1] / 16 + 1) * U * mag + 2.0 ** -8 * ref.abs()
                    assert bool(((got.double() - ref).abs() <= tol).all()), i
            del w
        dt = torch.bfloat16 if out == "bf16" else torch.float32
        for beta in (0.0, 1.0, 0.5):
            G = torch.full((e, n, k), 2.0, dtype=dt, device="cuda")
            mu.expert_grad(dy, x, off, G, beta=beta)
            assert mu.status()[0] == 0
            for i in counts:
                s = slice(o[i], o[i + 1])
                a, b = dy[s].double(), x[s].double()
                ref, mag = 2.0 * beta + a.T @ b, 2.0 * beta + a.abs().T @ b.abs()
                tol = 8 * U * mag + (2.0 ** -8 if out == "bf16" else U) * ref.abs()
                assert bool(((G[i].double() - ref).abs() <= tol).all()), (beta, i)
            for i in (1, 39, 41, e - 2):  # experts without rows, some of them behind 2^31
                assert bool((G[i] == 2.0 * beta).all()), (beta, i)
            del G
