"""Every plane product of the fp32 expert products counts (needs a B200).

fp32 operands are three bf16 planes, x = hi + mid + lo, and six products are kept: hi hi, hi mid, mid hi, mid mid,
hi lo, lo hi.  Where a row of the contraction holds one element other than zero, a result is that element's
product alone and errs by at most two units of 2^-23 for each of its six accumulations (adding zeros is
exact): 12 units, however long the contraction.  The values below put 32 units into every plane product but
hi hi, so that none may be missing or paired wrongly.
"""
import pytest

pytestmark = pytest.mark.gpu

U = 2.0 ** -23
VALUE = 1.0 + 2.0 ** -9 + 2.0 ** -18  # hi = 1, mid = 2^-9, lo = 2^-18
MID = 1.0 + 2.0 ** -9                 # squared: mid mid = 2^-18
# tokens an expert: split by the product kernel, packed, packed and paired
COUNTS = {"split": [5, 0, 64, 33], "packed": [70, 0, 300, 1], "paired": [2100, 0, 1031, 40]}


@pytest.fixture(scope="module")
def muon():
    from spectral_optimizer_state_b200 import Muon
    with Muon(0) as mu:
        yield mu


def _segments(counts):
    import torch
    o = [0]
    for c in counts:
        o.append(o[-1] + c)
    return torch.tensor(o, dtype=torch.int32, device="cuda"), o


def _values(shape, a, b):
    """a everywhere but in every third place, where b is, with signs and powers of two that change."""
    import torch
    n = 1
    for s in shape:
        n *= s
    i = torch.arange(n, device="cuda")
    v = torch.where(i % 3 == 0, b, a).double() * torch.where(i % 2 == 0, 1.0, -1.0).double() * torch.exp2(((i % 7) - 3).double())
    return v.reshape(shape).float()


def _permutation(rows, cols, shift):
    """[rows, cols] with one element other than zero a row: column (row + shift) % cols."""
    import torch
    m = torch.zeros(rows, cols, dtype=torch.float64, device="cuda")
    r = torch.arange(rows, device="cuda")
    m[r, (r + shift) % cols] = 1.0
    return m


def _close(got, ref):
    bad = (got.double() - ref).abs() > 12 * U * ref.abs()
    return not bool(bad.any())


@pytest.mark.parametrize("a,b", [(VALUE, 1.0), (1.0, VALUE), (MID, MID), (VALUE, VALUE)])
@pytest.mark.parametrize("counts", list(COUNTS))
@pytest.mark.parametrize("n,k", [(520, 515), (96, 1030), (700, 64)])
def test_products_keep_every_plane(muon, n, k, counts, a, b):
    """Weights with one element a row (forward) or a column (input gradient); a the tokens', b the weights'."""
    import torch
    off, o = _segments(COUNTS[counts])
    e = len(COUNTS[counts])
    one = torch.tensor(1.0, device="cuda")
    x, dy = _values((o[-1], k), one * a, one), _values((o[-1], n), one * a, one)
    scale = _values((e, n, k), one * b, one)
    forward = torch.stack([_permutation(n, k, 7 * i) for i in range(e)]) * scale.double()
    backward = torch.stack([_permutation(k, n, 5 * i).T for i in range(e)]) * scale.double()
    y, dx = muon.expert_matmul(x, forward.float(), off), muon.expert_matmul(dy, backward.float(), off, transpose=True)
    assert muon.status()[0] == 0
    for i in range(e):
        s = slice(o[i], o[i + 1])
        # the plane products left out (mid lo, lo lo) are below 2^-26 of the result
        assert _close(y[s], x[s].double() @ forward[i].T), ("forward", i)
        assert _close(dx[s], dy[s].double() @ backward[i]), ("input gradient", i)


@pytest.mark.parametrize("a,b", [(VALUE, 1.0), (1.0, VALUE), (MID, MID), (VALUE, VALUE)])
@pytest.mark.parametrize("counts", list(COUNTS))
@pytest.mark.parametrize("n,k", [(200, 328), (77, 129), (515, 3000)])
def test_gradients_keep_every_plane(muon, n, k, counts, a, b):
    """Only one token of a segment has values; a the gradient's, b the token's."""
    import torch
    off, o = _segments(COUNTS[counts])
    e = len(COUNTS[counts])
    one = torch.tensor(1.0, device="cuda")
    for place in (0, 1):  # the segment's first row, or its last
        dy, x = torch.zeros(o[-1], n, device="cuda"), torch.zeros(o[-1], k, device="cuda")
        live = [o[i] if place == 0 else o[i + 1] - 1 for i in range(e) if o[i + 1] > o[i]]
        dy[live], x[live] = _values((len(live), n), one * a, one), _values((len(live), k), one * b, one)
        G = muon.expert_grad(dy, x, off, torch.empty(e, n, k, device="cuda"))
        assert muon.status()[0] == 0
        for i in range(e):
            s = slice(o[i], o[i + 1])
            assert _close(G[i], dy[s].double().T @ x[s].double()), (place, i)


@pytest.mark.parametrize("k", [1, 5, 16, 17, 40, 100])
@pytest.mark.parametrize("counts", list(COUNTS))
def test_short_contractions_stay_sharp(muon, k, counts):
    """Random operands: six accumulations for every 16 elements, two units each, of the summed magnitudes; the
    products left out sum to at most 2^-21 of them; the parts' fp32 sums and the result a unit each."""
    import torch
    off, o = _segments(COUNTS[counts])
    e, n = len(COUNTS[counts]), 136
    g = torch.Generator(device="cuda")
    g.manual_seed(k)
    x, w = torch.randn(o[-1], k, generator=g, device="cuda"), torch.randn(e, n, k, generator=g, device="cuda")
    dy, wt = torch.randn(o[-1], k, generator=g, device="cuda"), torch.randn(e, k, n, generator=g, device="cuda")
    y, dx = muon.expert_matmul(x, w, off), muon.expert_matmul(dy, wt, off, transpose=True)
    rel = 2 * min(48, 6 * -(-k // 16)) * U + 2.0 ** -21 + 2 * U
    for i in range(e):
        s = slice(o[i], o[i + 1])
        for got, inp, m in ((y, x, w[i].T), (dx, dy, wt[i])):
            ref, mag = inp[s].double() @ m.double(), inp[s].double().abs() @ m.double().abs()
            assert bool(((got[s].double() - ref).abs() <= rel * mag).all()), i


@pytest.mark.parametrize("exponent", [-90, -105, -110, -114, -118, -122, -126, -130])
@pytest.mark.parametrize("counts", ["split", "packed"])
def test_values_near_the_bottom_of_the_range(muon, counts, exponent):
    """bf16 planes go no finer than 2^-133, so an operand below 2^-110 is held to 2^-134 instead of 2^-24 of itself;
    everything else is as above."""
    import torch
    off, o = _segments(COUNTS[counts])
    e, n, k = len(COUNTS[counts]), 72, 40
    g = torch.Generator(device="cuda")
    g.manual_seed(3)

    def draw(*shape, tiny):
        t = torch.randn(*shape, generator=g, device="cuda")
        return (t.double() * 2.0 ** exponent).float() if tiny else t

    def check(got, a, b, steps, what):
        """got = a @ b, a or b of them tiny."""
        a, b = a.double(), b.double()
        rel = 2 * min(48, steps) * U + 2.0 ** -21 + 2 * U
        held = 2.0 ** -134 * (a.abs().sum(1, keepdim=True) + b.abs().sum(0, keepdim=True)) + 2.0 ** -148
        assert bool(((got.double() - a @ b).abs() <= rel * (a.abs() @ b.abs()) + held).all()), what

    for tiny_rows in (True, False):
        x, dy = draw(o[-1], k, tiny=tiny_rows), draw(o[-1], n, tiny=tiny_rows)
        w, xg = draw(e, n, k, tiny=not tiny_rows), draw(o[-1], k, tiny=not tiny_rows)
        y, dx = muon.expert_matmul(x, w, off), muon.expert_matmul(dy, w, off, transpose=True)
        G = muon.expert_grad(dy, xg, off)
        assert muon.status()[0] == 0
        for i in range(e):
            s = slice(o[i], o[i + 1])
            check(y[s], x[s], w[i].T, 6 * -(-k // 16), ("forward", i))
            check(dx[s], dy[s], w[i], 6 * -(-n // 16), ("input gradient", i))
            check(G[i], dy[s].T, xg[s], 48, ("gradient", i))
