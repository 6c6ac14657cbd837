"""bf16 experts whose gradients micro-batches add to an fp32 buffer, through the Muon step (needs a B200)."""
import numpy as np
import pytest

import oracle
from tests.gpu_common import BF16_TOL, to_numpy

pytestmark = pytest.mark.gpu


def test_bf16_experts_with_a_main_gradient_are_stepped():
    """Two micro-batches, one stack as whole matrices and one by blocks, on the current stream and on another.
    The step's gradient is the buffer rounded to bf16; the step itself is within the bf16 bound of its oracle."""
    import torch
    from spectral_optimizer_state_b200 import Muon, expert_linear, torch_optimizer
    q5, hp = [oracle.QUINTIC] * 5, dict(lr=0.02, beta=0.95, weight_decay=0.1, eps=1e-7)
    off = torch.tensor([0, 50, 50, 140], dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    p = {"moe.in_proj": (0.05 * torch.randn(3, 160, 96, generator=g, device="cuda")).bfloat16().requires_grad_(),
         "moe.out_proj": (0.05 * torch.randn(3, 96, 160, generator=g, device="cuda")).bfloat16().requires_grad_()}
    main = {n: torch.zeros(t.shape, device="cuda") for n, t in p.items()}
    before = {n: to_numpy(t) for n, t in p.items()}
    opt = torch_optimizer(list(p.items()), stacked=True, blocks={"out_proj": (96, 64)}, main_grads=main)
    with Muon(0) as mu:
        for _ in range(2):
            x = torch.randn(140, 96, generator=g, device="cuda").bfloat16()
            h = torch.nn.functional.silu(expert_linear(x, p["moe.in_proj"], off, mu, grad_into=main["moe.in_proj"]))
            expert_linear(h, p["moe.out_proj"], off, mu, grad_into=main["moe.out_proj"]).square().sum().backward()
        assert mu.status()[0] == 0
    grads = {n: to_numpy(b.bfloat16()) for n, b in main.items()}
    assert all(t.grad is None for t in p.values()) and all(b.any() for b in main.values())
    opt.step()
    assert opt.inner.ctx.status()[0] == 0
    for n, cuts in (("moe.in_proj", [(0, 96)]), ("moe.out_proj", [(0, 64), (64, 128), (128, 160)])):
        got = to_numpy(p[n])
        for i in (0, 2):
            for c0, c1 in cuts:
                W, G = before[n][i][:, c0:c1], grads[n][i][:, c0:c1]
                ref = oracle.muon_step(W, G, np.zeros_like(G), q5, **hp)["W"]
                step = np.linalg.norm(ref - W * (1 - 0.02 * 0.1))
                err = np.linalg.norm(got[i][:, c0:c1] - ref)
                assert err <= BF16_TOL * step + 2.0 ** -8 * np.linalg.norm(ref), (n, i, c0)
        # an expert without tokens has a zero gradient: it only decays
        assert np.abs(got[1] - before[n][1] * (1 - 0.02 * 0.1)).max() <= 2.0 ** -8 * np.abs(before[n][1]).max()
    opt.zero_grad()
    assert not any(b.any() for b in main.values())
    # on a stream of the caller's, the rounded copies are made and freed there
    side = torch.cuda.Stream()
    twin = {n: t.detach().clone() for n, t in p.items()}
    from spectral_optimizer_state_b200 import MuonAdamW
    a = MuonAdamW(list(twin.items()), stacked=True, blocks={"out_proj": (96, 64)})
    b = MuonAdamW([(n, t.clone()) for n, t in twin.items()], stacked=True, blocks={"out_proj": (96, 64)})
    fresh = {n: torch.randn(t.shape, generator=g, device="cuda") for n, t in p.items()}
    torch.cuda.synchronize()
    for _ in range(3):
        a.step(fresh, stream=side)
        junk = [torch.full((3, 160, 96), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(4)]
        del junk
    side.synchronize()
    for _ in range(3):
        b.step({n: t.bfloat16() for n, t in fresh.items()})
    torch.cuda.synchronize()
    for x, y in zip(a.muon.values(), b.muon.values()):
        for (_, w, m), (_, wb, mb) in zip(x, y):
            assert torch.equal(w, wb) and torch.equal(m, mb)
    for o in (a, b, opt.inner):
        o.close()
