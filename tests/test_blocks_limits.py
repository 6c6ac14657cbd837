"""Which blocks the block calls take, and that the optimizer refuses others before anything is stepped (no GPU)."""
import ctypes

import pytest
import torch

from spectral_optimizer_state_b200 import MuonError, binding, optim
from spectral_optimizer_state_b200.build import build


@pytest.fixture(scope="module")
def lib():
    build()
    return binding.load_library()


class _Ctx:
    made = 0

    def __init__(self, *a, **k):
        type(self).made += 1
        self.calls = []

    def step_groups(self, *a, **k):
        self.calls.append("groups")

    def step_blocks(self, W, G, M, block, stream=None, **hp):
        self.calls.append(block)


@pytest.fixture()
def host(monkeypatch, lib):
    monkeypatch.setattr(optim, "Muon", _Ctx)
    monkeypatch.setattr(optim, "adamw_step", lambda *a, **k: None)
    _Ctx.made = 0


def test_documented_limits(lib):
    """128 for the shorter side; with it 5632 (bf16) and 2560 (fp32) for the longer, in either direction."""
    for dtype, most in ((0, 5632), (1, 2560)):
        for short in (113, 120, 128):
            assert lib.muon_check_blocks(short, most, short, most, dtype) == 0
            assert lib.muon_check_blocks(most, short, most, short, dtype) == 0
            assert lib.muon_check_blocks(short, most + 1, short, most + 1, dtype) == 2
            assert lib.muon_check_blocks(most + 1, short, most + 1, short, dtype) == 2
        for short in (1, 16, 64, 96, 112):  # no less for shorter ones
            assert lib.muon_check_blocks(short, most, short, most, dtype) == 0
            assert lib.muon_check_blocks(most, short, most, short, dtype) == 0
        assert lib.muon_check_blocks(4096, 4096, 129, 129, dtype) == 2
        assert lib.muon_check_blocks(4096, 4096, 4096, 1, dtype) == 0
        assert lib.muon_check_blocks(100, 90, 4096, 4096, dtype) == 0  # never larger than the matrix
    assert lib.muon_check_blocks(32769, 8, 8, 8, 0) == 2 and lib.muon_check_blocks(8, 32769, 8, 8, 0) == 2
    assert lib.muon_check_blocks(32768, 32768, 1, 1, 0) == 2  # more than 2^27 blocks
    for bad in ((0, 8, 8, 8), (8, 0, 8, 8), (8, 8, 0, 8), (8, 8, 8, -1)):
        assert lib.muon_check_blocks(*bad, 0) == 1
    assert lib.muon_check_blocks(8, 8, 8, 8, 7) == 3


@pytest.mark.parametrize("block", [(129, 129), (None, 129), (0, 64), (64, -1), (None, None)])
def test_blocks_that_cannot_be_stepped_are_refused_when_the_optimizer_is_made(host, block):
    p = [("a.in_proj", torch.zeros(256, 256)), ("b.in_proj", torch.zeros(256, 256))]
    with pytest.raises(MuonError):
        optim.MuonAdamW(p, blocks={"b.": block})
    with pytest.raises(MuonError):
        optim.MuonAdamW([("moe.in_proj", torch.zeros(2, 256, 256))], stacked=True, blocks={"moe": block})
    assert _Ctx.made == 0


def test_blocks_of_parameters_that_muon_does_not_take_are_not_looked_at(host):
    opt = optim.MuonAdamW([("a.in_proj", torch.zeros(256, 256)), ("emb", torch.zeros(200, 200))],
                          blocks={"emb": (200, 200), "a.": (64, None)})
    opt.step({"a.in_proj": torch.ones(256, 256)})
    assert opt.ctx.calls == [(64, None)]
    opt = optim.MuonAdamW([("a.out_proj", torch.zeros(256, 256))], mode="in_proj", blocks={"a.": (256, 256)})
    assert opt.muon_names() == []


def test_check_block_reads_sizes_as_step_blocks_does(lib):
    binding.check_block((100, 5000), (128, None), torch.bfloat16)  # the whole side where the block is larger
    binding.check_block((4096, 64), (None, 2 ** 40), torch.float32)
    with pytest.raises(MuonError) as e:
        binding.check_block((2 ** 33 + 64, 64), (64, 64), torch.float32)  # not taken modulo 2^32
    assert e.value.status == 2
    with pytest.raises(TypeError):
        binding.check_block((64, 64), (64, 64), torch.float16)
