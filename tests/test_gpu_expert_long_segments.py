"""bf16 weight gradients of segments far longer than an accumulator should sum (needs a B200)."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def muon():
    from spectral_optimizer_state_b200 import Muon
    with Muon(0) as mu:
        yield mu


def _same_sign(seed, tokens, cols):
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (0.5 + torch.rand(tokens, cols, generator=g, device="cuda")).to(torch.bfloat16)


def _reference(dy, x):
    import torch
    ref = torch.zeros(dy.shape[1], x.shape[1], dtype=torch.float64, device="cuda")
    for t in range(0, dy.shape[0], 1 << 17):
        ref += dy[t:t + (1 << 17)].double().T @ x[t:t + (1 << 17)].double()
    return ref


@pytest.mark.parametrize("beta,scale", [(0.0, 1.0), (1.0, 0.5)])
def test_a_long_sum_is_not_biased(muon, beta, scale):
    """2^20 tokens of one expert, all products positive.  Tensor-core additions truncate: by at most two units of
    2^-23 of the sum an addition of 16 products, so that one accumulator over the segment may lose 1.6e-2 of it
    (and loses about 65536 * 2^-24 * 0.7 = 2.7e-3, where a truncation costs half a unit on average), always
    towards zero.  Summed by 32768 tokens, as many elements as a product contracts at most, the loss is at most
    2 * 2048 * 2^-23 of the whole, the fp32 sums of the 32 parts err by 2^-24 each.  Rounding to bf16 errs by at most 2^-8 with no bias: over 256 x 256
    elements the mean of their relative errors lies within six times 2^-8 / sqrt(3 * 65536) of zero."""
    import torch
    tokens, n, k = 1 << 20, 256, 256
    x, dy = _same_sign(1, tokens, k), _same_sign(2, tokens, n)
    off = torch.tensor([0, 0, tokens, tokens], dtype=torch.int32, device="cuda")
    G = torch.ones(3, n, k, dtype=torch.bfloat16, device="cuda")
    muon.expert_grad(dy, x, off, G, beta=beta, scale=scale)
    assert muon.status()[0] == 0
    ref = scale * _reference(dy, x) + beta
    rel = (G[1].double() - ref) / ref
    lost = 2 * 2048 * 2.0 ** -23 + 33 * 2.0 ** -24
    assert abs(float(rel.mean())) <= lost + 6 * 2.0 ** -8 / (3 * 65536) ** 0.5
    assert float(rel.abs().max()) <= lost + 2.0 ** -8
    want = torch.full_like(G[0], beta)  # experts without rows
    assert torch.equal(G[0], want) and torch.equal(G[2], want)


@pytest.mark.parametrize("tokens", [32768, 32769, 32832, 65536, 80001])
def test_segments_around_a_part(muon, tokens):
    """Long and short segments of one call, odd sizes, rows of another expert behind the long one."""
    import torch
    for n, k in ((72, 200), (77, 129), (1, 3), (300, 136)):
        x, dy = _same_sign(3, tokens + 50, k), _same_sign(4, tokens + 50, n)
        x[1::2].neg_()
        x[tokens:] *= 100.0
        off = torch.tensor([0, tokens, tokens, tokens + 50], dtype=torch.int32, device="cuda")
        for out in (torch.bfloat16, torch.float32):
            G = torch.full((3, n, k), float("nan"), dtype=out, device="cuda")
            muon.expert_grad(dy, x, off, G)
            assert muon.status()[0] == 0 and not G[1].any()
            for e, (a, b) in ((0, (0, tokens)), (2, (tokens, tokens + 50))):
                ref, mag = _reference(dy[a:b], x[a:b]), _reference(dy[a:b], x[a:b].abs())
                # truncation within a part, the fp32 sums of the parts, the result's rounding
                tol = (2 * 2048 * 2.0 ** -23 + 5 * 2.0 ** -24) * mag + (2.0 ** -8 if out == torch.bfloat16 else 2.0 ** -23) * ref.abs()
                assert bool(((G[e].double() - ref).abs() <= tol).all()), (n, k, out, e)
