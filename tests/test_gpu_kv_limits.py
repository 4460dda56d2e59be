"""Attention calls as large as their arguments may be: more blocks than a launch holds, more entries than a workgroup has
threads, prompts and long single tokens in one call."""
from __future__ import annotations

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from _kv import UNIT, Pair, np64  # noqa: E402
from test_gpu_kv_attend import run  # noqa: E402
from oracle import kv_oracle as KO  # noqa: E402
import bit_weight_only_packed_amd as Q  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _gpu_present():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def test_more_blocks_than_a_launch_holds():
    """1,024 entries of up to 2,000 rows and 1,024 kv heads: 2^24 blocks of 256 threads, of which two entries have any."""
    n = heads = 1024
    kv = Q.KVCache(16, 16, heads, 64, max_seqs=n, max_pages=8)
    kv.pool.normal_(generator=torch.Generator("cuda").manual_seed(1))
    grow = torch.zeros(n, dtype=torch.int32)
    grow[5], grow[1000] = 40, 70
    kv.extend(grow.cuda())
    kv.check()
    q = torch.empty((2048, heads, 64), dtype=torch.float16, device="cuda").normal_(generator=torch.Generator("cuda").manual_seed(2))
    start = torch.zeros(n + 1, dtype=torch.int32)
    start[6:1001], start[1001:] = 2000, 2048
    print("2^24 blocks", flush=True)
    out = kv.attend(q, seqs=torch.arange(n, dtype=torch.int32).cuda(), row_start=start.cuda(), max_rows=2000)
    torch.cuda.synchronize()
    for slot, a, b, length in ((5, 0, 2000, 40), (1000, 2000, 2048, 70)):
        alone = kv.attend(q[a:b], seqs=torch.tensor([slot], dtype=torch.int32).cuda())
        assert torch.equal(alone.view(torch.int16), out[a:b].view(torch.int16))
        t = kv.pool[kv.tables[slot, :-(-length // 16)].long(), 0].transpose(0, 1)  # [2][pages][heads][16][64]
        for h in (0, 511, 1023):
            k, v = (np64(t[i][:, h]).reshape(-1, 64)[:length] for i in (0, 1))
            for r in (a, b - 30, b - 1):
                x = np64(q[r, h])
                ref = KO.attend_row(x, k, v, length - (b - r), 0.125)
                u = UNIT["f16"]
                es = 66 * 2.0 ** -24 * np.abs(x).sum() * np.abs(k).max() * 0.125
                tol = np.abs(v).max() * (u + 2 * es + (length + 64) * 2.0 ** -23) + u * np.abs(ref) + 2.0 ** -24
                assert (np.abs(np64(out[r, h]) - ref) <= tol).all()


@pytest.mark.parametrize("n,D,rows,G", [(257, 256, 1, 2), (512, 64, 2, 2), (513, 128, 1, 1), (700, 64, 1, 3), (1024, 64, 1, 1),
                                        (600, 64, 5, 7)])
def test_entries_past_the_threads_of_a_workgroup(n, D, rows, G):
    """The list of entries is made in several passes: 256 or 512 at a time (the last case: the many-row kernel)."""
    lens = [(29 * i) % 70 for i in range(n)]
    slots = [int(s) for s in np.random.default_rng(n).permutation(n)]
    run(Pair(lens, "f16", 16, 1, D), [rows] * n, G, slots=slots, uniform=True)


@pytest.mark.parametrize("D,dtype", [(64, "f16"), (128, "bf16"), (256, "f16")])
def test_prompts_and_long_single_tokens_in_one_call(D, dtype):
    """A chunk of a prompt beside decoding slots, some far longer than it, and an idle one."""
    run(Pair([200, 9001, 3, 0, 2500, 170], dtype, 32, 2, D), [140, 1, 1, 1, 1, 0], 3)
    run(Pair([9001, 200, 3, 0, 70], dtype, 32, 1, D), [1, 140, 3, 1, 70], 4, window=700, sinks=5)
