"""What calls on the cache refuse, leave out or leave alone."""
from __future__ import annotations

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from _kv import Pair, check_out, np64, rand  # noqa: E402
import bit_weight_only_packed_amd as Q  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _gpu_present():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def ints(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("n_new", [[1, 1, 40, 1], [1, 1, 200, 1]], ids=["short", "long"])
@pytest.mark.parametrize("rows", [1, 3])
def test_append_after_a_refused_extend_writes_nothing(n_new, rows):
    """The tokens that the slots hold, shared ones among them, stay as they were; the next extend that is granted, or
    bits that the caller has cleared, let rows in again."""
    p = Pair([20, 33, 5], "f16", 16, 2, 64, extra=2, spare_slots=1, max_pages=8)
    p.gpu.fork([0], [3])
    p.ref.fork([0], [3])
    k, v = rand((4 * rows, 2, 64), "f16", 5), rand((4 * rows, 2, 64), "f16", 6)
    seqs = ints(0, 1, 2, 3)
    before = p.gpu.pool.clone()
    p.gpu.extend(n_new)
    p.gpu.append(k, v, seqs=seqs)
    assert torch.equal(before.view(torch.int16), p.gpu.pool.view(torch.int16))
    p.same_state()
    # a step that is granted: its rows are written
    p.gpu.extend([0, 0, rows, 0])
    p.ref.extend([0, 0, rows, 0])
    p.gpu.append(k[:rows], v[:rows], seqs=ints(2))
    p.ref.append(0, [2], [rows], np64(k[:rows]), np64(v[:rows]))
    p.same_state()
    # refused again, then looked at: the caller may write over the last tokens as ever
    p.gpu.extend(n_new)
    with pytest.raises(Q.QGError):
        p.gpu.check()
    p.gpu.append(k[:rows], v[:rows], seqs=ints(1))
    p.ref.append(0, [1], [rows], np64(k[:rows]), np64(v[:rows]))
    p.same_state()


def test_captured_steps_that_run_out_of_pages():
    """Replays of a captured step past the last free page: lengths, tables and every stored token stay."""
    p = Pair([30, 14], "f16", 16, 2, 64, extra=1, max_pages=6)
    k, v = rand((2, 2, 64), "f16", 5), rand((2, 2, 64), "f16", 6)
    one, seqs = ints(1, 1), ints(0, 1)

    def step():
        p.gpu.extend(one)
        p.gpu.append(k, v, seqs=seqs)

    step()
    p.ref.extend([1, 1])
    p.ref.append(0, [0, 1], [1, 1], np64(k), np64(v))
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for i in range(5):  # the second of these needs two pages
        k.copy_(rand(k.shape, "f16", 100 + i))
        g.replay()
        p.ref.extend([1, 1])
        p.ref.append(0, [0, 1], [1, 1], np64(k), np64(v))
        p.same_state()
    assert p.ref.info[0] and p.gpu.lens.tolist() == [32, 16]


@pytest.mark.parametrize("most", [1, 3, 16, 40])
def test_rows_past_max_rows_are_left_out(most):
    """The others stand where they would: at len - R + i with all R rows counted, through both kernels."""
    lens, rows, slots = [70, 9, 130], [50, 9, 41], [0, 1, 2]
    p = Pair(lens, "f16", 16, 2, 64)
    n, start = sum(rows), [0] + list(np.cumsum(rows))
    k, v, q = rand((n, 2, 64), "f16", 5), rand((n, 2, 64), "f16", 6), rand((n, 4, 64), "f16", 7, 1.5)
    kw = dict(seqs=ints(*slots), row_start=ints(*start), max_rows=most)
    off = [r for a, b in zip(start, start[1:]) for r in range(a + most, b)]
    for window, sinks in ((0, 0), (8, 2)):
        ref = p.ref.attend(0, slots, rows, np64(q), 0.125, window, sinks)
        out = torch.full_like(q, 7.0)
        p.gpu.attend(q, window=window, sinks=sinks, out=out, **kw)
        assert (out[off] == 7).all()
        out[off] = torch.from_numpy(ref[off]).half().cuda()
        check_out(out, ref, "f16", q, p, 0, slots, rows, 0.125)
    p.gpu.append(k, v, **kw)
    p.ref.append(0, slots, rows, np64(k), np64(v), max_rows=most)
    p.same_state()


def test_rows_past_max_rows_before_the_start():
    """Rows that are left out count for the position also where that is before the first token."""
    p = Pair([5, 40], "f16", 16, 1, 64)
    q = rand((90, 2, 64), "f16", 7)
    for most in (8, 40):
        out = p.gpu.attend(q, seqs=ints(0, 1), row_start=ints(0, 45, 90), max_rows=most, out=torch.full_like(q, 7.0))
        o = np64(out)
        assert (o[:most] == 0).all()  # positions -40 ..
        assert (o[45:50] == 0).all() and (o[50:45 + most] != 0).any(axis=(1, 2)).all()  # positions -5 ..
        assert (o[most:45] == 7).all() and (o[45 + most:] == 7).all()


@pytest.mark.parametrize("n_new", [[50, 0, 0], [1000, 7, 900], [0, 33, 0], [1 << 22, 1 << 22, 1 << 22]])
def test_extend_says_how_many_pages_are_short(n_new):
    """Also where one slot wants more than the whole pool."""
    p = Pair([20, 3, 0], "f16", 16, 1, 64, extra=1, max_pages=1 << 20)
    p.gpu.fork([0], [2])
    p.ref.fork([0], [2])
    p.gpu.extend(n_new)
    p.ref.extend(n_new)
    p.same_state()
    assert p.gpu.info.tolist()[:2] == p.ref.info[:2] and p.ref.info[1] > 0
    assert p.ref.info[1] > (3 * (1 << 18) - 2 if n_new[2] > 1000 else 0)


@pytest.mark.parametrize("given", [False, True])
def test_check_waits_for_work_on_other_streams(given):
    """An extend that is refused late, on a stream of its own, is found, and its bits are gone when check returns."""
    kv = Q.KVCache(2, 16, 1, 64, max_seqs=1, max_pages=4)
    n = ints(50)
    for _ in range(2):
        s, other = torch.cuda.Stream(), torch.cuda.Stream()
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            torch.cuda._sleep(100_000_000)
        kv.extend(n, stream=s)
        with pytest.raises(Q.QGError, match="2 free pages short"):
            kv.check(stream=s if given else None)
        with torch.cuda.stream(other):
            assert kv.info.tolist()[:2] == [0, 0]
        kv.check()


@pytest.mark.parametrize("rows", [2, 70])
def test_outputs_that_overlap_are_refused(rows):
    """out over itself or over q, whole or in part; not where they only lie between each other."""
    p = Pair([rows + 30], "f16", 16, 2, 64)
    q = rand((rows, 4, 64), "f16", 7, 1.5)
    kw = dict(seqs=ints(0))
    want = p.gpu.attend(q, **kw)
    store = torch.zeros(rows * 1024, dtype=torch.float16, device="cuda")

    def view(row, head, ofs=0):
        return store[ofs:].as_strided((rows, 4, 64), (row, head, 1))

    for row, head in ((64, 64), (128, 64), (192, 64), (64, 128), (320, 128), (0, 64), (256, 32), (256, 0), (256, 64),
                      (264, 64), (64, 64 * rows), (640, 192), (1024, 256)):
        places = [r * row + h * head + e for r in range(rows) for h in range(4) for e in range(0, 64, 8)]
        if len(set(places)) < len(places):
            with pytest.raises(Q.QGError, match="overlap"):
                p.gpu.attend(q, out=view(row, head), **kw)
        else:
            assert torch.equal(want, p.gpu.attend(q, out=view(row, head), **kw))
    for row, head, ofs in ((256, 64, 0), (256, 64, 8), (256, 64, 256), (512, 64, 224), (1024, 128, 32), (512, 128, 128)):
        store.zero_()
        x = view(row, head)
        x.copy_(q)
        with pytest.raises(Q.QGError, match="out overlaps q"):
            p.gpu.attend(x, out=view(row, head, ofs), **kw)
        assert torch.equal(x, q)
    for row, head, ofs in ((512, 64, 256), (512, 128, 64), (1024, 128, 64), (1024, 192, 64), (256, 64, 256 * rows)):
        store.zero_()
        x = view(row, head)
        x.copy_(q)
        assert torch.equal(want, p.gpu.attend(x, out=view(row, head, ofs), **kw)) and torch.equal(x, q)


def test_steps_without_rows():
    """A call of no rows does nothing, whatever its entries."""
    p = Pair([20, 33], "f16", 16, 2, 64)
    kv = torch.empty((0, 2, 64), dtype=torch.float16, device="cuda")
    q = torch.empty((0, 4, 64), dtype=torch.float16, device="cuda")
    for kw in (dict(), dict(seqs=[]), dict(seqs=[1]), dict(seqs=ints(0, 1)), dict(row_start=[0], max_rows=0),
               dict(seqs=[1, 0], row_start=ints(0, 0, 0), max_rows=0), dict(seqs=[0], row_start=[0, 0], max_rows=5)):
        p.gpu.append(kv, kv, **kw)
        assert p.gpu.attend(q, **kw).shape == (0, 4, 64)
    p.same_state()
    for bad in (dict(layer=1), dict(seqs=[0, 1, 1])):
        with pytest.raises(Q.QGError):
            p.gpu.append(kv, kv, **bad)
        with pytest.raises(Q.QGError):
            p.gpu.attend(q, **bad)
    one = rand((1, 2, 64), "f16", 5)
    with pytest.raises(Q.QGError):
        p.gpu.append(one, one, seqs=[])


@pytest.mark.parametrize("heads,rows", [(1, 5), (2, 1), (1, 1), (1, 40), (2, 40)])
def test_strides_of_a_single_row_or_head_are_not_used(heads, rows):
    """They may be anything, as a slice's are; those that are used are held to their rule."""
    p, same = (Pair([60], "f16", 16, heads, 64) for _ in range(2))
    q, k, v = rand((rows, 2 * heads, 64), "f16", 3), rand((rows, heads, 64), "f16", 4), rand((rows, heads, 64), "f16", 5)
    kw = dict(seqs=ints(0))

    def odd(x):
        row, head = (3 if rows == 1 else x.stride(0)), (5 if x.shape[1] == 1 else x.stride(1))
        return x.as_strided(x.shape, (row, head, 1))

    same.gpu.append(k, v, **kw)
    p.gpu.append(odd(k), odd(v), **kw)
    assert torch.equal(p.gpu.pool.view(torch.int16), same.gpu.pool.view(torch.int16))
    out = odd(torch.empty_like(q))
    assert torch.equal(p.gpu.attend(odd(q), out=out, **kw), same.gpu.attend(q, **kw))
    if heads == 1:  # a single q head too
        one = odd(q[:, :1].contiguous())
        assert torch.equal(p.gpu.attend(one, **kw), same.gpu.attend(q[:, :1].contiguous(), **kw))
    wide = torch.zeros(rows * 1024 + 1024, dtype=torch.float16, device="cuda")
    with pytest.raises(Q.QGError, match="strides"):
        p.gpu.attend(wide.as_strided((rows, 2 * heads, 64), (1000, 68, 1)), **kw)
    if rows > 1:
        with pytest.raises(Q.QGError, match="strides"):
            p.gpu.append(wide.as_strided((rows, heads, 64), (1004, 64, 1)), v, **kw)
