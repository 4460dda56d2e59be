"""Calls of attend_shared that share nothing, or not for every entry: where the plan turns sharing down the call is
attend bit for bit, in both kernels and with blocks that several workgroups share."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from _kv import rand  # noqa: E402
from test_gpu_kv_shared import Forked, ints  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _gpu_present():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("D,heads,G,rows", [(64, 1, 20, 2), (128, 2, 20, 2), (128, 1, 5, 40), (256, 1, 12, 2), (256, 2, 4, 9),
                                            (64, 2, 4, 1), (128, 1, 5, 3), (256, 1, 8, 1)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (1500, 4)])
def test_turned_down_by_the_plan(dtype, D, heads, G, rows, window, sinks):
    """Prompts of 2,000 tokens, of which 1,984 are shared, and a limit one token above them: the plan runs and says no."""
    f = Forked([2000], [[43, 60, 70]], dtype, 16, heads, D, seed=20)
    token = 4 * heads * D
    q = rand((3 * rows, heads * G, D), dtype, 16, 1.5)
    kw = dict(seqs=ints(0, 1, 2), window=window, sinks=sinks)
    least = 3 * (min(1984, window + sinks) if window else 1984) * token + token
    got = f.gpu.attend_shared(q, least=least, **kw)
    assert torch.equal(got, f.gpu.attend(q, **kw))
    f.check(q, got, [0, 1, 2], [rows] * 3, window, sinks, dtype)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("D,G", [(64, 20), (128, 20), (256, 12)])
def test_an_entry_that_shares_nothing_beside_a_group(dtype, D, G):
    """Many rows of a kv head: the lone entry's bits are those of attend."""
    f = Forked([2000, 1900], [[43, 60, 70], [50]], dtype, 16, 1, D, seed=21)
    q = rand((8, G, D), dtype, 17, 1.5)
    kw = dict(seqs=ints(0, 1, 2, 3))
    got = f.gpu.attend_shared(q, groups=ints(0, 3, 4), **kw)
    f.check(q, got, [0, 1, 2, 3], [2] * 4, dtype=dtype)
    plain = f.gpu.attend(q, **kw)
    assert torch.equal(got[6:], plain[6:]) and not torch.equal(got[:6], plain[:6])
