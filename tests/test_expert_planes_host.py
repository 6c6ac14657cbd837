"""The plane tests of the fp32 expert products would see a missing or a wrong plane product (no GPU: a model of the
six products in fp64)."""
import numpy as np
import pytest

from synthetic import round_bf16
from tests.test_gpu_expert_planes import MID, U, VALUE

PAIRS = [(1, 1), (0, 2), (2, 0), (0, 1), (1, 0), (0, 0)]  # plane 0 = hi, 1 = mid, 2 = lo


def _planes(v):
    out, rest = [], np.float64(v)
    for _ in range(3):
        out.append(float(np.ravel(round_bf16(np.array([rest], np.float32)))[0]))
        rest -= out[-1]
    assert rest == 0.0
    return out


def _product(a, b, pairs):
    pa, pb = _planes(a), _planes(b)
    return sum(pa[i] * pb[j] for i, j in pairs)


CASES = [(VALUE, 1.0), (1.0, VALUE), (MID, MID), (VALUE, VALUE)]


def test_all_six_products_are_exact_enough():
    for a, b in CASES:
        assert abs(_product(a, b, PAIRS) - a * b) <= 2.0 ** -26 * a * b


@pytest.mark.parametrize("missing", PAIRS)
def test_a_missing_product_is_outside_the_bound(missing):
    kept = [p for p in PAIRS if p != missing]
    assert any(abs(_product(a, b, kept) - a * b) > 12 * U * a * b for a, b in CASES)


@pytest.mark.parametrize("place,wrong", [(p, (i, j)) for p in range(6) for i in range(3) for j in range(3) if PAIRS[p] != (i, j)])
def test_a_product_of_other_planes_is_outside_the_bound(place, wrong):
    pairs = PAIRS[:place] + [wrong] + PAIRS[place + 1:]
    assert any(abs(_product(a, b, pairs) - a * b) > 12 * U * a * b for a, b in CASES)
