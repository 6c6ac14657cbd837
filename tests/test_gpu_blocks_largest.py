"""The longest blocks that the block calls take, against the fp64 oracle (needs a B200)."""
import numpy as np
import pytest

import oracle
from tests.gpu_common import BF16_TOL, F32_TOL, to_numpy

pytestmark = pytest.mark.gpu

Q5 = [oracle.QUINTIC] * 5
# shorter side, longest wide block, longest tall block
LARGEST = {"bf16": [(128, 5632, 5632), (112, 6144, 5632), (65, 9728, 6144), (64, 13312, 13312), (16, 32768, 13312), (1, 32768, 13312)],
           "f32": [(128, 2560, 2560), (96, 3584, 2560), (65, 4096, 2560), (64, 6144, 6144), (17, 12800, 6144), (1, 26112, 6144)]}


@pytest.mark.parametrize("dtype,shape", [(d, s) for d, ls in LARGEST.items() for m, w, t in ls for s in ((m, w), (t, m))])
def test_the_longest_blocks(dtype, shape):
    import torch
    from spectral_optimizer_state_b200 import Muon, binding
    dt, code = (torch.bfloat16, 0) if dtype == "bf16" else (torch.float32, 1)
    longer = tuple(n + 1 if n == max(shape) else n for n in shape)
    check = binding.load_library().muon_check_blocks
    assert check(*shape, *shape, code) == 0 and check(*longer, *longer, code) == 2
    g = torch.Generator(device="cuda")
    g.manual_seed(sum(shape))
    X = [torch.randn(*shape, generator=g, device="cuda").to(dt) for _ in range(2)]
    Out = [torch.full_like(x, float("nan")) for x in X]
    with Muon(0, coeffs=Q5) as mu:
        mu.orthogonalize_blocks(X, Out, shape)
        assert mu.status() == (0, [0, 0])
    half, tol = (2.0 ** -8, BF16_TOL) if dtype == "bf16" else (2.0 ** -24, F32_TOL)
    for x, o in zip(X, Out):
        ref, _ = oracle.orthogonalize(to_numpy(x), Q5, eps=1e-7)
        assert np.linalg.norm(to_numpy(o) - ref) <= (tol + half) * np.linalg.norm(ref)
