"""Sampling of as many rows as a call may have."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import bit_weight_only_packed_amd as Q  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _gpu_present():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


@pytest.mark.parametrize("rows", [2 ** 22 + 1, 2 ** 31 - 1])
def test_as_many_rows_as_there_may_be(rows):
    """One row's logits for all of them: every token is written, those of the last launch too, and nothing behind them."""
    x = torch.tensor([[-1.0]], dtype=torch.float16, device="cuda")
    u = torch.zeros(rows, device="cuda")
    out = torch.full((rows + 64,), -7, dtype=torch.int32, device="cuda")
    Q.sample(x.expand(rows, 1), u, temperature=0.0, out=out[:rows])
    torch.cuda.synchronize()
    for at in range(0, rows, 1 << 28):  # (a piece at a time: reductions of whole tensors take 32-bit counts)
        piece = out[at:min(at + (1 << 28), rows)]
        assert int(piece.min()) == 0 and int(piece.max()) == 0
    assert (out[rows:] == -7).all()
