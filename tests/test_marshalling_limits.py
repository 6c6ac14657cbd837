"""Sizes that do not fit the library's 32-bit fields are refused, not taken modulo 2^32 (no GPU)."""
import pytest
import torch

from spectral_optimizer_state_b200 import MuonError, binding


class _Lib:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, args))
            return 0
        return call


@pytest.fixture()
def host(monkeypatch):
    """A Muon whose tensors may live on the CPU and whose library only records."""
    mu = object.__new__(binding.Muon)
    mu.lib, mu.handle, mu.device = _Lib(), None, -1
    monkeypatch.setattr(mu, "_device_stream", lambda s: 0, raising=False)
    return mu


def _expanded(*shape, dtype=torch.float32):
    """A tensor of any size with one element of memory."""
    return torch.zeros(1, dtype=dtype).expand(1).as_strided(shape, (0,) * len(shape))


@pytest.mark.parametrize("shape", [(2 ** 32 + 5, 1, 1), (5, 2 ** 32 + 1, 1), (5, 1, 2 ** 32 + 1)])
def test_expert_calls(host, shape):
    tokens, n, k = shape
    off = torch.tensor([0, 2, 5], dtype=torch.int32)
    x, dy, w = _expanded(tokens, k), _expanded(tokens, n), _expanded(2, n, k)
    for call in (lambda: host.expert_matmul(x, w, off), lambda: host.expert_matmul(dy, w, off, transpose=True),
                 lambda: host.expert_grad(dy, x, off)):
        with pytest.raises(MuonError) as e:
            call()
        assert e.value.status == 2
    assert host.lib.calls == []


@pytest.mark.parametrize("shape,block", [((2 ** 32 + 8, 4), (8, 4)), ((4, 2 ** 32 + 8), (4, 8))])
def test_block_calls_of_long_matrices(host, monkeypatch, shape, block):
    monkeypatch.setattr(torch.Tensor, "is_cuda", property(lambda t: True))
    host.device = None
    t = _expanded(*shape)
    with pytest.raises(MuonError) as e:
        host.orthogonalize_blocks([t], [t], block)
    assert e.value.status == 2 and host.lib.calls == []


@pytest.mark.parametrize("block,want", [((2 ** 32 + 2, 4), (6, 4)), ((4, 2 ** 40 + 3), (4, 8)), ((-2 ** 32 + 2, 4), (0, 4)),
                                        ((-3, 4), (0, 4)), ((None, 100), (6, 8))])
def test_block_sizes_beyond_32_bits(host, monkeypatch, block, want):
    """A block larger than the matrix is the whole side; one that is not positive reaches the library as such."""
    monkeypatch.setattr(torch.Tensor, "is_cuda", property(lambda t: True))
    host.device = None
    host.orthogonalize_blocks([torch.zeros(6, 8)], [torch.zeros(6, 8)], block)
    b = host.lib.calls[0][1][1]._obj
    assert (b.block_rows, b.block_cols) == want


def test_no_matrices_are_refused_like_other_bad_lists(host):
    for W in ([], torch.zeros(0, 6, 8)):
        with pytest.raises(ValueError):
            host.orthogonalize_blocks(W, W, (3, 8))
        with pytest.raises(ValueError):
            host.block_step_plan(W, W, W, (3, 8))
    assert host.lib.calls == []
