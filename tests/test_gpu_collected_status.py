"""Errors of expert and block calls are kept until muon_get_status reports them, whatever the context does in
between: steps of whole matrices, other block calls, reading the norms, graphs (needs a B200)."""
import pytest

pytestmark = pytest.mark.gpu

HP = dict(lr=0.02, beta=0.95, weight_decay=0.1, eps=1e-7)


@pytest.fixture()
def muon():
    from spectral_optimizer_state_b200 import Muon
    with Muon(0) as mu:
        yield mu


def _matrices(rows=64, cols=96, nan=False):
    import torch
    t = [[0.02 * torch.randn(rows, cols, device="cuda")] for _ in range(3)]
    if nan:
        t[1][0][40, 5] = float("nan")
    return t


def _experts():
    import torch
    x, w = torch.ones(10, 64, dtype=torch.bfloat16, device="cuda"), torch.ones(3, 72, 64, dtype=torch.bfloat16, device="cuda")
    good = torch.tensor([0, 4, 4, 10], dtype=torch.int32, device="cuda")
    bad = torch.tensor([0, 5, 3, 10], dtype=torch.int32, device="cuda")
    return x, w, good, bad


def _status(muon):
    """The status code, whether it comes back or is raised."""
    from spectral_optimizer_state_b200 import MuonError
    try:
        return muon.status()[0]
    except MuonError as e:
        return e.status


def test_bad_offsets_outlive_a_step_of_whole_matrices(muon):
    x, w, good, bad = _experts()
    muon.expert_matmul(x, w, bad)
    muon.step(*_matrices(), **HP)
    muon.expert_matmul(x, w, good)
    assert _status(muon) == 1
    assert _status(muon) == 0  # reported once


def test_a_flagged_block_outlives_later_calls(muon):
    muon.step_blocks(*_matrices(nan=True), (32, 96), **HP)
    muon.step_blocks(*_matrices(), (32, 96), **HP)
    st, flags = muon.status()
    assert st == 5 and flags == [0, 0]  # the flags are the last call's
    assert muon.status() == (0, [0, 0])
    muon.step_blocks(*_matrices(nan=True), (32, 96), **HP)
    muon.step(*_matrices(), **HP)
    assert muon.status() == (5, [0])
    assert muon.status() == (0, [0])
    muon.step_blocks(*_matrices(nan=True), (32, 96), **HP)
    assert muon.status() == (5, [0, 1])


def test_an_optimizer_step_reports_its_blocks_and_the_products_before_it():
    import torch
    from spectral_optimizer_state_b200 import MuonAdamW
    p = {"heads.in_proj": torch.randn(64, 96, device="cuda"), "whole.in_proj": torch.randn(48, 96, device="cuda")}
    opt = MuonAdamW(list(p.items()), blocks={"heads": (32, None)})
    g = {n: torch.randn_like(t) for n, t in p.items()}
    opt.step(g)
    assert opt.ctx.status()[0] == 0
    g["heads.in_proj"][3, 3] = float("inf")
    opt.step(g)
    assert opt.ctx.status()[0] == 5
    x, w, good, bad = _experts()
    opt.ctx.expert_matmul(x, w, bad)
    g["heads.in_proj"][3, 3] = 0.0
    opt.step({"whole.in_proj": g["whole.in_proj"]})
    assert _status(opt.ctx) == 1 and _status(opt.ctx) == 0
    opt.close()


def test_norms_do_not_take_the_status(muon):
    x, w, good, bad = _experts()
    muon.expert_matmul(x, w, bad)
    muon.step_blocks(*_matrices(), (32, 96), **HP)
    assert len(muon.norms()) == 2
    muon.expert_matmul(x, w, good)
    assert muon.norms() == []
    assert _status(muon) == 1 and _status(muon) == 0


def test_replays_report_what_happened_since_the_last_report(muon):
    import torch
    x, w, good, bad = _experts()
    off, y = good.clone(), torch.zeros(10, 72, dtype=torch.bfloat16, device="cuda")
    muon.expert_matmul(x, w, bad)
    assert _status(muon) == 1
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):  # an error has just been read
        muon.expert_matmul(x, w, off, out=y)

    def replay(o):
        off.copy_(o)
        graph.replay()
        torch.cuda.synchronize()

    replay(good)
    assert _status(muon) == 0
    replay(bad)
    replay(good)
    assert _status(muon) == 1  # the second replay did not wipe it
    replay(good)
    assert _status(muon) == 0  # and it is not reported again
    replay(bad)
    assert _status(muon) == 1
    del graph


def test_an_empty_call_reports_nothing_of_the_call_before(muon):
    import torch
    x, w, good, bad = _experts()
    muon.step_blocks(*_matrices(), (32, 96), **HP)
    muon.expert_matmul(x[:0], w, torch.zeros_like(good))
    assert muon.status() == (0, []) and muon.norms() == []


def test_a_step_from_host_gradients_reports_its_own_matrices(muon):
    """Its result is its own; what a product before it reported stays for status()."""
    import torch
    x, w, good, bad = _experts()
    muon.expert_matmul(x, w, bad)
    W, G, M = _matrices()
    nu, flags = muon.step_groups_host([(W, [G[0].cpu().pin_memory()], M)], **HP)
    assert flags == [0] and nu[0] > 0
    assert _status(muon) == 1 and _status(muon) == 0
    torch.cuda.synchronize()
