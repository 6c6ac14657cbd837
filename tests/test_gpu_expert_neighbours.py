"""Expert products and gradients write their outputs and nothing beside them: views with elements of others to the
left, to the right and between the rows, at every width and start (needs a B200)."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def muon():
    from spectral_optimizer_state_b200 import Muon
    with Muon(0) as mu:
        yield mu


def _dt(name):
    import torch
    return torch.bfloat16 if name == "bf16" else torch.float32


COUNTS = {"few": [0, 5, 40], "many": [100, 0, 333, 90]}


def _offsets(counts):
    import torch
    o = [0]
    for c in counts:
        o.append(o[-1] + c)
    return torch.tensor(o, dtype=torch.int32, device="cuda"), o


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("counts", list(COUNTS))
@pytest.mark.parametrize("width", [1, 3, 5, 29, 31, 33, 49, 64, 127, 130, 171, 300])
def test_products(muon, width, counts, dtype):
    import torch
    off, o = _offsets(COUNTS[counts])
    e, k, dt = len(o) - 1, 40, _dt(dtype)
    x, w = torch.randn(o[-1], k, device="cuda").to(dt), torch.randn(e, width, k, device="cuda").to(dt)
    want = muon.expert_matmul(x, w, off)
    wt = w.transpose(1, 2).contiguous()  # the same product as an input gradient
    for ld in sorted({width, width + 1, -(-width // 4) * 4, -(-width // 8) * 8, -(-width // 8) * 8 + 8}):
        for start in (0, 1, 4, 8):
            buf = torch.full((o[-1] + 2, ld + start), 7.0, dtype=dt, device="cuda")
            out = buf[1:-1, start:start + width]
            muon.expert_matmul(x, w, off, out=out)
            assert torch.equal(out, want)
            out.fill_(7.0)
            assert bool((buf == 7.0).all()), (ld, start)
            muon.expert_matmul(x, wt, off, transpose=True, out=out)
            out.fill_(7.0)
            assert bool((buf == 7.0).all()), (ld, start)


@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("counts", list(COUNTS))
@pytest.mark.parametrize("rows,width", [(1, 1), (1, 49), (16, 5), (17, 31), (33, 33), (40, 49), (130, 127), (20, 171), (64, 300)])
def test_gradients(muon, rows, width, counts, dtype, out):
    import torch
    off, o = _offsets(COUNTS[counts])
    e = len(o) - 1
    dy, x = (torch.randn(o[-1], c, device="cuda").to(_dt(dtype)) for c in (rows, width))
    for beta in (0.0, 1.0, 0.5):
        want = muon.expert_grad(dy, x, off, torch.ones(e, rows, width, dtype=_dt(out), device="cuda"), beta=beta)
        for ld in sorted({width, -(-width // 4) * 4, -(-width // 8) * 8 + 8}):
            for start in (0, 1, 4):
                buf = torch.full((e, rows + 2, ld + start), float("nan"), dtype=_dt(out), device="cuda")
                G = buf[:, 1:-1, start:start + width]
                G.fill_(1.0)
                muon.expert_grad(dy, x, off, G, beta=beta)
                # beta = 1 may be added up by the memory system, at some strides and not at others: one more rounding
                assert torch.allclose(G.float(), want.float(), rtol=2.0 ** -7 if out == "bf16" else 2.0 ** -22, atol=1e-6), (ld, start)
                G.fill_(float("nan"))
                assert bool(buf.isnan().all()), (beta, ld, start)


def test_one_row_of_a_flat_buffer(muon):
    """Gradients of a single row, or matrix, that lie side by side in one buffer."""
    import torch
    off = torch.tensor([0, 20], dtype=torch.int32, device="cuda")
    dy, x = torch.randn(20, 1, device="cuda"), torch.randn(20, 49, device="cuda")
    for beta in (0.0, 1.0):
        flat = torch.full((256,), float("nan"), device="cuda")
        G = flat[64:64 + 49].view(1, 1, 49)
        G.fill_(0.0)
        muon.expert_grad(dy, x, off, G, beta=beta)
        assert not bool(G.isnan().any()) and bool(flat[:64].isnan().all()) and bool(flat[64 + 49:].isnan().all())
        flat = torch.full((256,), 7.0, device="cuda")
        muon.expert_grad(dy, x, off, flat[64:64 + 49].view(1, 1, 49), beta=beta)
        assert bool((flat[:64] == 7.0).all()) and bool((flat[64 + 49:] == 7.0).all())
