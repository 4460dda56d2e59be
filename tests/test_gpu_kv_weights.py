"""The weights of the attention where they are hard to hold: far below the largest, and of scores so large that their
last bits are worth many powers of two."""
from __future__ import annotations

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from _kv import DT, UNIT, np64  # noqa: E402
import bit_weight_only_packed_amd as Q  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _gpu_present():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("slots,rows,G", [(32, 1, 1), (1, 136, 64)], ids=["few", "many"])
@pytest.mark.parametrize("gap", [12.0, 16.0, 17.5])
def test_weights_far_below_the_largest(dtype, slots, rows, G, gap):
    """Eight tokens with values of 0 take nearly all the weight; the 65,000 others, exp(-gap) of it each, make the
    output.  Enough (entry, head) pairs and blocks that their tokens are not shared out: the tokens that a wave goes
    through hang on the largest."""
    T, heads, D, page = 65537, 8, 64, 256
    rng = np.random.default_rng(int(gap))
    s = torch.from_numpy(rng.uniform(-1, 1, T)).to(DT[dtype])
    s[:256:32] = gap
    val = torch.from_numpy(rng.uniform(0.5, 1, (T, D))).to(DT[dtype])
    val[:256:32] = 0
    need = -(-T // page)
    pool = torch.zeros((need, 1, 2, heads, page, D), dtype=DT[dtype])
    pad = need * page - T
    pool[:, 0, 0, :, :, 0] = torch.nn.functional.pad(s, (0, pad)).view(need, 1, page)
    pool[:, 0, 1] = torch.nn.functional.pad(val, (0, 0, 0, pad)).view(need, 1, page, D)
    tables = torch.arange(need, dtype=torch.int32).expand(slots, need).contiguous().cuda()
    kv = Q.KVCache.of(pool.cuda(), tables, torch.full((slots,), T, dtype=torch.int32).cuda(),
                      torch.full((need,), slots, dtype=torch.int32).cuda())
    q = torch.zeros((slots * rows, heads * G, D), dtype=DT[dtype], device="cuda")
    q[:, :, 0] = 8  # times the scale of 1/8: the scores are the keys' first elements, exactly
    out = np64(kv.attend(q, seqs=torch.arange(slots, dtype=torch.int32, device="cuda"))).reshape(slots, rows, heads * G, D)
    w = np.exp(np64(s) - gap)
    num, den = np.cumsum(w[:, None] * np64(val), 0), np.cumsum(w)
    at = np.arange(T - rows, T)
    ref = np.broadcast_to((num[at] / den[at, None])[None, :, None], out.shape)
    u = UNIT[dtype]
    err = np.abs(out - ref)
    rms = float(np.sqrt(np.mean(err ** 2)) / np.sqrt(np.mean(ref ** 2)))
    print("gap", gap, "ref", ref.flat[0], "out", out.flat[0], "rms", rms, flush=True)
    assert (err <= u + (T + 64) * 2.0 ** -23 + u * ref + 2.0 ** -24).all()
    assert rms <= 2 * u


@pytest.mark.parametrize("dtype,size", [("f16", 3000.0), ("f16", 54656.0), ("f16", 61280.0), ("f16", 64896.0),
                                        ("bf16", 216 * 2.0 ** 43), ("bf16", 221 * 2.0 ** 43)])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("rows,G", [(1, 3), (100, 2)])
def test_equal_scores_of_any_size_give_the_mean(rows, G, D, sign, dtype, size):
    """Weights of one value whatever the scores (sizes whose product with scale log2(e) is rounded by up to 2^5, and in
    bf16 by 2^74, either way); one token below them takes no part."""
    T, page = 300, 32
    need = -(-T // page)
    g = torch.Generator().manual_seed(D)
    pool = torch.zeros((need, 1, 2, 2, page, D), dtype=DT[dtype])
    low = 0.5 * size if sign > 0 else size  # times q: below the others
    pool[:, 0, 0, :, :, 1] = size if sign > 0 else 0.5 * size
    pool[0, 0, 0, :, 7, 1] = low
    pool[:, 0, 1] = torch.rand((need, 2, page, D), generator=g, dtype=torch.float64).to(DT[dtype])
    kv = Q.KVCache.of(pool.cuda(), torch.arange(need, dtype=torch.int32)[None].cuda(), torch.tensor([T], dtype=torch.int32).cuda(),
                      torch.ones(need, dtype=torch.int32).cuda())
    q = torch.zeros((rows, 2 * G, D), dtype=DT[dtype], device="cuda")
    q[:, :, 1] = sign * size
    out = np64(kv.attend(q, seqs=torch.zeros(1, dtype=torch.int32, device="cuda")))
    v = np64(pool[:, 0, 1]).transpose(1, 0, 2, 3).reshape(2, need * page, D)[:, :T]
    u = UNIT[dtype]
    for i in range(rows):
        seen = np.arange(T - rows + i + 1)
        ref = v[:, seen[seen != 7]].mean(1).repeat(G, 0)
        assert (np.abs(out[i] - ref) <= u + (T + 64) * 2.0 ** -23 + u * ref).all()
