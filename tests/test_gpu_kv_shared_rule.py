"""Which route attend_shared takes by itself: the one that was measured to be the faster, on both sides of the limits
(where it is attend its bits are attend's, where tokens are shared they are not)."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from _kv import UNIT, rand  # noqa: E402
import bit_weight_only_packed_amd as Q  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _gpu_present():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


# q heads, kv heads, head size, rows, entries, shared tokens; us of attend and with shared tokens
@pytest.mark.parametrize("qh,kvh,D,rows,n,prompt,shares", [
    (16, 2, 256, 1, 64, 4096, False),   # 57 / 89: 512 MiB
    (16, 2, 256, 1, 64, 8192, False),   # 83 / 100
    (16, 2, 256, 1, 16, 32768, True),   # 157 / 111
    (16, 2, 256, 8, 64, 8192, False),   # 221 / 271
    (40, 8, 128, 4, 64, 2048, False),   # 60 / 92: 512 MiB
    (40, 8, 128, 1, 64, 8192, True),    # 130 / 82
    (32, 4, 128, 4, 64, 8192, False),   # 78 / 108: 1 GiB
    (8, 8, 64, 1, 64, 8192, True),      # 85 / 55
    (64, 8, 64, 4, 64, 4096, False),    # 64 / 87: 512 MiB
    (64, 8, 64, 4, 64, 8192, False),    # 98 / 111: 1 GiB
])
def test_the_route_by_default(qh, kvh, D, rows, n, prompt, shares):
    page = 64
    kv = Q.KVCache(prompt // page + 3 * n, page, kvh, D, max_seqs=n + 1, max_pages=prompt // page + 3, dtype=torch.bfloat16)
    kv.pool.normal_(generator=torch.Generator("cuda").manual_seed(1))
    kv.extend([0] * n + [prompt])
    kv.fork([n] * n, list(range(n)))
    kv.extend([100] * n + [0])
    kv.check()
    q = rand((n * rows, qh, D), "bf16", 2)
    seqs = torch.arange(n, dtype=torch.int32, device="cuda")
    got, plain = kv.attend_shared(q, seqs=seqs), kv.attend(q, seqs=seqs)
    assert torch.equal(got, plain) != shares
    # both are within 2 u of the definition in the root mean square
    err = (got.double() - plain.double()).square().mean().sqrt()
    assert err <= 4 * UNIT["bf16"] * plain.double().square().mean().sqrt()
