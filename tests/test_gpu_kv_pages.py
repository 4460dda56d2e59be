"""Page operations and the append against the oracle: every table, length, count
and pool bit equal."""
from __future__ import annotations

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from _kv import Pair, np64, rand  # noqa: E402
import bit_weight_only_packed_amd as Q  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _gpu_present():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def both(p, op, *args):
    print(op, [list(a)[:12] if a is not None else None for a in args], flush=True)
    getattr(p.gpu, op)(*args)
    getattr(p.ref, op)(*args)
    p.same_state()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("page", [16, 64])
def test_append(dtype, D, page):
    lens, rows = [1, 16, 17, 100, 0, 65, 3], [1, 16, 5, 100, 2, 0, 7]   # rows past a slot's start are left out
    p = Pair(lens, dtype, page, 3, D, layers=2)
    start = [0] + list(np.cumsum(rows))
    qkv = rand((sum(rows), 11, D), dtype, 5)
    k, v = qkv[:, 5:8], qkv[:, 8:]
    slots = [3, 0, 2, 1, 6, 5, 4]
    rows = [min(r, 200) for r in rows]
    p.gpu.append(k, v, layer=1, seqs=slots, row_start=start, max_rows=100)
    p.ref.append(1, slots, rows, np64(k), np64(v))
    p.same_state()


def test_append_uniform_and_bad_pages():
    p = Pair([40, 40], "f16", 16, 2, 64)
    k, v = rand((8, 2, 64), "f16", 1), rand((8, 2, 64), "f16", 2)
    p.gpu.append(k, v)
    # without seqs, rows / n with n = min(rows, slots): slots 0 and 1, four rows each
    p.ref.append(0, [0, 1], [4, 4], np64(k), np64(v))
    p.same_state()
    # a table entry that names no page is not written through
    p.gpu.tables[1, 2] = 1 << 29
    before = p.gpu.pool.clone()
    p.gpu.append(k[:4] + 1, v[:4] + 1, seqs=[1])
    assert torch.equal(before, p.gpu.pool)


@pytest.mark.parametrize("layers", [1, 3])
def test_fork_extend_trim_compact(layers):
    """The life of a few sequences, every step compared."""
    p = Pair([5, 33, 48, 1], "f16", 16, 2, 64, layers=layers, extra=40, spare_slots=6, max_pages=10)
    both(p, "fork", [0, 1, 1, 2], [4, 5, 6, 7])
    both(p, "extend", [1, 0, 0, 0, 0, 0, 0, 0, 0, 0])          # 0 leaves the shared tail to 4
    both(p, "extend", [0, 1, 0, 0, 2, 1, 1, 1, 0, 20])         # all three of 1, 5, 6 grow: the lowest keeps the page
    both(p, "extend", [0, 0, 1, 15, 0, 0, 0, 0, 0, -4])
    both(p, "trim", [5, 1], [20, 40])
    both(p, "fork", [5], [8])
    both(p, "extend", [0, 0, 0, 0, 0, 1, 0, 0, 0, 0])
    both(p, "trim", [0, 7, 3])
    both(p, "compact")
    both(p, "extend", [30, 1, 1, 1, 1, 1, 1, 1, 1, 1])
    both(p, "compact")
    both(p, "trim", list(range(10)))
    both(p, "compact")
    p.gpu.check()
    assert int(p.gpu.refs.sum()) == 0


@pytest.mark.parametrize("seed", range(4))
def test_random_lives(seed):
    rng = np.random.default_rng(seed)
    p = Pair([int(n) for n in rng.integers(0, 60, 6)], "bf16", 16, 1, 64, extra=30, spare_slots=5, max_pages=9, seed=seed)
    for _ in range(25):
        op = rng.choice(["extend", "extend", "fork", "trim", "compact"])
        if op == "extend":
            both(p, op, [int(n) for n in rng.integers(0, 5, 11)])
        elif op == "fork":
            both(p, op, [int(n) for n in rng.integers(-1, 12, 3)], [int(n) for n in rng.integers(-1, 12, 3)])
        elif op == "trim":
            both(p, op, [int(n) for n in rng.integers(-1, 12, 2)], [int(n) for n in rng.integers(-3, 50, 2)])
        else:
            both(p, op)
    bits = int(p.gpu.info[0])
    assert bits == p.ref.info[0]


@pytest.mark.parametrize("pages", [1, 3, 4095, 4096, 4097, 9001])
def test_compact_many_pages(pages):
    """Free lists over several passes of the deciding workgroup, and counts that are no multiple of four."""
    rng = np.random.default_rng(pages)
    n = max(1, pages // 3)
    ids = rng.permutation(pages)[:n]
    pool = torch.arange(pages, dtype=torch.float32).to(torch.bfloat16).view(pages, 1, 1, 1, 1, 1)
    pool = pool.expand(pages, 1, 2, 1, 16, 64).contiguous().cuda()
    tables = torch.from_numpy(ids.astype(np.int32)).view(1, -1).cuda()
    refs = torch.zeros(pages, dtype=torch.int32)
    refs[torch.from_numpy(ids)] = 1
    kv = Q.KVCache.of(pool, tables, torch.tensor([n * 16], dtype=torch.int32).cuda(), refs.cuda())
    before = pool[tables[0].long()].clone()
    kv.compact()
    assert sorted(kv.tables[0].tolist()) == list(range(n))
    assert torch.equal(kv.pool[kv.tables[0].long()], before)
    assert kv.refs.tolist() == [1] * n + [0] * (pages - n)
    assert kv.info.tolist()[2:] == [n, int((ids >= n).sum())]
    same = kv.tables.clone()
    kv.compact()
    assert torch.equal(same, kv.tables) and kv.info.tolist()[3] == 0


def test_extend_takes_many_pages_at_once():
    kv = Q.KVCache(6000, 16, 1, 64, max_seqs=1000, max_pages=4000)
    n = torch.zeros(1000, dtype=torch.int32)
    n[3], n[700], n[999] = 50001, 17, 1
    kv.extend(n.cuda())
    kv.check()
    assert kv.tables[3, :3126].tolist() == list(range(3126)) and int(kv.tables[3, 3126]) == -1
    assert kv.tables[700, :2].tolist() == [3126, 3127] and kv.tables[999, 0] == 3128
    assert kv.lens[[3, 700, 999]].tolist() == [50001, 17, 1] and int(kv.refs.sum()) == 3129


def test_extend_is_all_or_nothing():
    p = Pair([16, 16], "f16", 16, 1, 64, extra=2, max_pages=3)
    both(p, "extend", [17, 17])                 # two pages each, two free
    with pytest.raises(Q.QGError, match="2 free pages short"):
        p.gpu.check()
    p.gpu.check()
    both(p, "extend", [33, 0])                  # a table of three entries
    with pytest.raises(Q.QGError, match="longer"):
        p.gpu.check()
    both(p, "extend", [2 ** 31 - 1, 2 ** 31 - 1])
    with pytest.raises(Q.QGError):
        p.gpu.check()
    both(p, "extend", [16, 16])
    p.gpu.check()


def test_fork_and_trim_refuse_entries():
    p = Pair([20, 30], "f16", 16, 1, 64, spare_slots=3)
    both(p, "fork", [0, 0, 1, 9, 2], [2, 2, 0, 3, 4])
    with pytest.raises(Q.QGError, match="refused"):
        p.gpu.check()
    both(p, "trim", [1, 1, -1, 5], [3, 0, 0, 0])
    with pytest.raises(Q.QGError, match="refused"):
        p.gpu.check()


def test_refusals():
    kv = Q.KVCache(8, 16, 2, 64, max_seqs=2)
    with pytest.raises(ValueError):
        kv.extend([1])
    with pytest.raises(ValueError):
        kv.fork([0, 1], [1])
    with pytest.raises(Q.QGError):
        kv.trim([0, 1, 0])
    with pytest.raises(Q.QGError):
        kv.trim([])
    k = rand((1, 2, 64), "f16", 1)
    with pytest.raises(ValueError):
        kv.append(k, k[:, :1])
    with pytest.raises(Q.QGError):
        kv.append(k, k, layer=1)
    with pytest.raises(Q.QGError):
        Q.KVCache(8, 24, 2, 64)
    with pytest.raises(Q.QGError):
        Q.KVCache(8, 16, 2, 96)
    with pytest.raises(Q.QGError):
        Q.KVCache(8, 16, 2, 64, max_seqs=1025)
    with pytest.raises(TypeError):
        Q.KVCache(8, 16, 2, 64, dtype=torch.float32)
    with pytest.raises(ValueError):
        Q.KVCache.of(kv.pool, kv.tables.long(), kv.lens, kv.refs)
    with pytest.raises(ValueError):
        Q.KVCache.of(kv.pool, kv.tables, kv.lens, kv.refs[:4])
    with pytest.raises(ValueError):
        Q.KVCache.of(kv.pool.transpose(3, 4), kv.tables, kv.lens, kv.refs)
