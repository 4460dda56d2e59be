"""The norm at the ends of its number formats, against the definition in fp64."""
from __future__ import annotations

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from _kv import UNIT, np64  # noqa: E402
from oracle import step_oracle as SO  # noqa: E402
import bit_weight_only_packed_amd as Q  # noqa: E402

TINY = 2.0 ** -149  # fp32's smallest number


@pytest.fixture(scope="module", autouse=True)
def _gpu_present():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


@pytest.mark.parametrize("n", [96, 4096, 20000])
@pytest.mark.parametrize("exp", [-70, -75])
def test_small_elements_beside_large_ones(n, exp):
    """A row whose squares pass fp32 because of one element: the others, 2^140 or more below it, keep the bits that fp32
    has for h / sqrt(mean), and a weight brings them back."""
    g = torch.Generator().manual_seed(n)
    x = (torch.rand((3, n), generator=g, dtype=torch.float64) + 1) * 2.0 ** exp
    x[:, 5] = 2.0 ** 70
    x, w = x.to(torch.bfloat16).cuda(), torch.full((n,), 2.0 ** 60, dtype=torch.bfloat16, device="cuda")
    y = Q.rms_norm(x, w)
    ref = SO.rms_norm(np64(x), np64(w))
    # the output's rounding, the arithmetic of the mean and root, and half of fp32's smallest number times the weight
    assert (np.abs(np64(y) - ref) <= np.abs(ref) * (UNIT["bf16"] + 40 * 2.0 ** -24) + TINY / 2 * 2.0 ** 60).all()
