"""Block calls refuse matrices that one block would read while another writes them (needs a B200)."""
import pytest

pytestmark = pytest.mark.gpu

HP = dict(lr=0.02, beta=0.95, weight_decay=0.1, eps=1e-7)


@pytest.fixture(scope="module")
def muon():
    from spectral_optimizer_state_b200 import Muon
    with Muon(0) as mu:
        yield mu


def _randn(seed, *shape):
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda")


def _refused(call):
    from spectral_optimizer_state_b200 import MuonError
    with pytest.raises(MuonError) as e:
        call()
    return e.value.status == 1


def test_outputs_that_are_inputs_of_other_matrices_are_refused(muon):
    a, b, c = (_randn(s, 64, 96) for s in (1, 2, 3))
    kept = [t.clone() for t in (a, b, c)]
    block = (32, 96)
    assert _refused(lambda: muon.orthogonalize_blocks([a, b], [b, a], block))
    assert _refused(lambda: muon.orthogonalize_blocks([a, b, c], [a, c, b], block))
    assert _refused(lambda: muon.step_blocks([a, b], [b, b], [c, _randn(4, 64, 96)], block, **HP))
    assert all(bool((x == y).all()) for x, y in zip((a, b, c), kept))


def test_momentum_that_is_a_weight_or_a_gradient_is_refused(muon):
    a, b, c, d = (_randn(s, 64, 96) for s in (1, 2, 3, 4))
    kept = [t.clone() for t in (a, b, c, d)]
    block = (32, 96)
    assert _refused(lambda: muon.step_blocks([a], [b], [a], block, **HP))
    assert _refused(lambda: muon.step_blocks([a], [b], [b], block, **HP))
    assert _refused(lambda: muon.step_blocks([a, b], [c, c], [d, a], block, **HP))
    assert _refused(lambda: muon.step_blocks([a, b], [c, d], [d, _randn(5, 64, 96)], block, **HP))
    assert all(bool((x == y).all()) for x, y in zip((a, b, c, d), kept))


def test_in_place_takes_the_same_stride(muon):
    import torch
    wide = _randn(6, 64, 192)
    half = wide.view(128, 96)[:64]  # the same address, another stride
    kept = wide.clone()
    assert _refused(lambda: muon.orthogonalize_blocks([wide[:, :96]], [half], (32, 96)))
    assert _refused(lambda: muon.step_blocks([half], [wide[:, :96]], [_randn(7, 64, 96)], (32, 96), **HP))
    assert bool((wide == kept).all())
    # one row has no stride
    row, want = _randn(8, 1, 96), torch.empty(1, 96, device="cuda")
    muon.orthogonalize_blocks([row], [want], (1, 48))
    muon.orthogonalize_blocks([row.as_strided((1, 96), (500, 1))], [row], (1, 48))
    assert torch.equal(row, want)
    # and the step may read its gradient from its own weights
    w, twin = wide[:, :96], wide[:, :96].clone()
    m, mt = _randn(9, 64, 96), _randn(9, 64, 96)
    muon.step_blocks([twin], [twin.clone()], [mt], (32, 96), **HP)
    muon.step_blocks([w], [w], [m], (32, 96), **HP)
    assert torch.equal(w, twin) and torch.equal(m, mt) and muon.status()[0] == 0
