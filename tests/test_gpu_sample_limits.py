"""Sampling at the ends of its number formats, by one workgroup a row and by parts, against the definition in fp64."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_sample import compare, draws  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _gpu_present():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("vocab", [5, 3001, 70001])
@pytest.mark.parametrize("settings", [dict(), dict(top_k=3), dict(top_p=0.9), dict(top_k=2000, top_p=0.97), dict(min_p=0.2),
                                      dict(top_k=4, top_p=0.8, min_p=0.05)])
def test_logits_farther_apart_than_fp32(dtype, vocab, settings):
    """Logits of both signs near fp32's largest, at temperatures as large: their difference passes fp32, their weights are
    ordinary numbers."""
    g = torch.Generator().manual_seed(vocab)
    x = ((torch.rand((4, vocab), generator=g, dtype=torch.float64) * 2 - 1) * 3.2e38).to(dtype)
    x[0, 1], x[0, 3] = 3e38, -3e38
    x[3] = torch.where(x[3] > 0, 3e38, -3e38).to(dtype)
    x = x.cuda()
    u = torch.tensor([0.95, 0.2, 0.6, 0.99]).cuda()
    for heat in (3e38, 1e38, 2e37, 1e30):
        compare(x, u, heat, **settings)
    compare(x, draws(4, vocab), torch.tensor([3e38, float("inf"), 1e37, 2e38]).cuda(), **settings)


@pytest.mark.parametrize("vocab", [5, 3001, 70001])
@pytest.mark.parametrize("settings", [dict(), dict(top_k=3), dict(top_p=0.9), dict(top_k=2000, top_p=0.97, min_p=0.01)])
def test_logits_closer_together_than_fp32_can_divide(vocab, settings):
    """Logits of some 10^-38 at temperatures as small, one over which passes fp32."""
    g = torch.Generator().manual_seed(vocab)
    x = (torch.randn((4, vocab), generator=g, dtype=torch.float64) * 1e-38).float().cuda()
    for heat in (1e-39, 1e-38, 1e-37, 1e-36, 2.0 ** -149):
        compare(x, draws(4, vocab + 1), heat, **settings)
