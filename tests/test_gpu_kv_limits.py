"""Attention calls as large as their arguments may be: more blocks than a launch holds, more entries than a workgroup has
threads, prompts and long single tokens in one call, pools
past 4 GiB, windows past any length."""
from __future__ import annotations

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from _kv import UNIT, Pair, np64, rand  # noqa: E402
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


@pytest.mark.parametrize("D,page", [(64, 16), (128, 64), (256, 32)])
def test_pools_past_four_gib(D, page):
    """Every operation on pages whose bytes and elements lie past 2^32, against the same on a small pool."""
    lens, heads, layers = [300, 47, 3], 2, 2
    small = Pair(lens, "f16", page, heads, D, layers=layers, extra=6, spare_slots=1, max_pages=40)
    gpu = small.gpu
    page_bytes = layers * 2 * heads * page * D * 2
    pages = (9 << 30) // page_bytes
    shift = pages - small.gpu.pages
    assert shift * page_bytes > 2 ** 33 and pages <= 1 << 20
    pool = torch.empty((pages,) + tuple(gpu.pool.shape[1:]), dtype=torch.float16, device="cuda")
    pool[shift:] = gpu.pool
    tables = torch.where(gpu.tables >= 0, gpu.tables + shift, gpu.tables)
    refs = torch.ones(pages, dtype=torch.int32, device="cuda")  # the pages below are taken
    refs[shift:] = gpu.refs
    big = Q.KVCache.of(pool, tables, gpu.lens.clone(), refs)
    seqs = torch.arange(3, dtype=torch.int32, device="cuda")

    def same():
        assert torch.equal(big.pool[shift:].view(torch.int16), gpu.pool.view(torch.int16))
        assert torch.equal(torch.where(big.tables >= 0, big.tables - shift, big.tables), gpu.tables)
        assert torch.equal(big.lens, gpu.lens) and torch.equal(big.refs[shift:], gpu.refs)

    def both(op, *args, **kw):
        print(op, flush=True)
        getattr(big, op)(*args, **kw)
        getattr(gpu, op)(*args, **kw)
        same()

    both("fork", [1], [3])
    both("extend", [1, 2, 40, 0])  # copies a shared tail
    for rows in (1, 40):
        k, v = rand((3 * rows, heads, D), "f16", 5), rand((3 * rows, heads, D), "f16", 6)
        both("append", k, v, layer=1, seqs=seqs)
        q = rand((3 * rows, 2 * heads, D), "f16", 7)
        a, b = (x.attend(q, layer=1, seqs=seqs) for x in (big, gpu))
        assert torch.isfinite(b).all() and torch.equal(a.view(torch.int16), b.view(torch.int16))
    big.trim([1])
    big.refs[2] = 0
    live = big.refs > 0
    m = int(live.sum())  # the live pages past it move, in order, into the free ones before it
    moved, to = torch.nonzero(live[m:])[:, 0] + m, torch.nonzero(~live[:m])[:, 0]
    assert moved.numel() == to.numel() > 0 and int(to[0]) == 2
    before = big.pool[moved].clone()
    big.compact()
    assert torch.equal(big.pool[to].view(torch.int16), before.view(torch.int16))


@pytest.mark.parametrize("rows", [1, 70])
def test_windows_and_sinks_past_any_length(rows):
    p = Pair([rows + 50, 3], "f16", 16, 2, 64)
    q = rand((2 * rows, 4, 64), "f16", 7)
    seqs = torch.arange(2, dtype=torch.int32, device="cuda")
    want = p.gpu.attend(q, seqs=seqs)
    top = 2 ** 31 - 1
    for window, sinks in ((top, 0), (top, top), (0, top), (1, top), (1 << 30, 3)):
        out = np64(p.gpu.attend(q, seqs=seqs, window=window, sinks=sinks))
        assert np.abs(out - np64(want)).max() <= 2 * UNIT["f16"] * float(p.gpu.pool.abs().max())
