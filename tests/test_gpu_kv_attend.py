"""Attention over the paged cache against the fp64 oracle: single tokens, verify
rows and prompts; heads, types, page sizes, ragged lengths, windows and sinks,
rows that see nothing, and non-finite values where a row does not look."""
from __future__ import annotations

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from _kv import DT, Pair, check_out, np64, rand  # noqa: E402
import bit_weight_only_packed_amd as Q  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _gpu_present():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def starts(rows):
    return [0] + list(np.cumsum(rows))


def attend(p, rows, G, *, slots=None, window=0, sinks=0, scale=None, seed=9, uniform=False):
    heads, D = p.gpu.kv_heads, p.gpu.head_dim
    slots = list(range(len(rows))) if slots is None else slots
    q = rand((sum(rows), heads * G, D), p.dtype, seed, 1.5)
    print("attend", p.dtype, "D", D, "heads", heads, "G", G, "page", p.gpu.page_size, "rows", rows[:8], "lens",
          p.ref.lens[:8], "window", window, sinks, flush=True)
    sc = D ** -0.5 if scale is None else scale
    kw = dict(window=window, sinks=sinks, scale=scale)
    if uniform:
        out = p.gpu.attend(q, seqs=slots, **kw)
    else:
        out = p.gpu.attend(q, seqs=slots, row_start=starts(rows), max_rows=max(max(rows), 1), **kw)
    torch.cuda.synchronize()
    ref = p.ref.attend(0, slots, rows, np64(q), sc, window, sinks)
    return q, out, ref, slots, sc


def run(p, rows, G, **kw):
    q, out, ref, slots, sc = attend(p, rows, G, **kw)
    check_out(out, ref, p.dtype, q, p, 0, slots, rows, sc)
    return out


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("page", [16, 64])
def test_one_token(dtype, D, page):
    """One new token of each slot at lengths around tiles and pages, an idle slot among them."""
    lens = [1, 2, 15, 16, 17, 0, 31, 32, 33, 64, 65, 127, 129, 257]
    run(Pair(lens, dtype, page, 2, D), [1] * len(lens), 5, uniform=True)


@pytest.mark.parametrize("G", [1, 2, 3, 7, 16, 17, 32])
def test_groups(G):
    run(Pair([5, 70, 200], "f16", 32, 3, 64), [1, 1, 1], G)


@pytest.mark.parametrize("heads", [1, 5, 8])
@pytest.mark.parametrize("page", [32, 128, 256])
def test_heads_and_pages(heads, page):
    run(Pair([3, 300], "bf16", page, heads, 128), [1, 1], 2)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("R,G", [(2, 5), (4, 4), (8, 4), (8, 5), (8, 8), (13, 5), (16, 8), (32, 5), (3, 64)])
def test_verify_rows(D, R, G):
    """Verify batches over both kernels (up to 32 or 16 rows of a kv head, and more)."""
    run(Pair([R, R + 1, 50 + R, 301], "f16", 16, 2, D), [R] * 4, G, uniform=True)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_ragged_prompts(dtype, D):
    """Prompts of many lengths, some behind a history, some with no rows at all."""
    lens = [1, 40, 129, 130, 257, 77, 0, 200]
    rows = [1, 40, 129, 3, 200, 0, 0, 64]
    run(Pair(lens, dtype, 16, 2, D), rows, 3)


@pytest.mark.parametrize("D", [64, 128])
def test_long_prompt_split(D):
    """Few blocks over many tokens: several workgroups share a block."""
    run(Pair([1500], "f16", 16, 1, D), [70], 2)


@pytest.mark.parametrize("rows", [1, 6, 90])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (5, 2), (16, 0), (33, 4), (64, 40), (100, 7), (1000, 3), (7, 500)])
def test_windows_and_sinks(rows, window, sinks):
    run(Pair([rows, 100 + rows, 260, 301], "f16", 16, 2, 64), [rows] * 4, 2, window=window, sinks=sinks)


@pytest.mark.parametrize("window,sinks", [(20, 3), (130, 0)])
def test_windows_wide_heads(window, sinks):
    run(Pair([400, 33], "bf16", 32, 1, 256), [1, 1], 8, window=window, sinks=sinks)
    run(Pair([400, 140], "bf16", 32, 1, 256), [140, 70], 2, window=window, sinks=sinks)


@pytest.mark.parametrize("rows", [4, 100])
def test_rows_before_the_start_see_nothing(rows):
    """More rows than tokens: the first rows stand at negative positions."""
    p = Pair([2, 0, 30], "f16", 16, 2, 128)
    out = run(p, [rows] * 3, 2, window=8, sinks=1)
    o = np64(out).reshape(3, rows, -1)
    assert (o[0, :rows - 2] == 0).all() and (o[1] == 0).all()


@pytest.mark.parametrize("scale", [1e-6, 1.0, 4.0])
def test_scale(scale):
    run(Pair([90, 10], "f16", 16, 2, 64), [1, 1], 2, scale=scale)
    run(Pair([90, 40], "f16", 16, 2, 64), [90, 40], 2, scale=scale)


@pytest.mark.parametrize("junk", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("rows,window,sinks", [(1, 0, 0), (5, 0, 0), (100, 0, 0), (1, 9, 2), (100, 9, 2)])
def test_memory_without_tokens(junk, rows, window, sinks):
    """Slots of pages past a sequence's length, and free pages, hold anything."""
    run(Pair([rows, 30 + rows, 105], "f16", 16, 2, 64, fill=junk), [rows] * 3, 3, window=window, sinks=sinks)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("rows", [6, 150])
@pytest.mark.parametrize("which", [0, 1])
def test_non_finite_tokens(D, dtype, rows, which):
    """A token whose key or value is not finite reaches the rows that see it and no other."""
    p = Pair([rows + 20], dtype, 16, 1, D)
    at = {rows + 20 - 3: float("nan"), rows + 20 - 2: -float("inf"), 25: float("inf")}
    for t, x in at.items():
        page = int(p.ref.tables[0, t // 16])
        p.gpu.pool[page, 0, which, 0, t % 16, 3] = x
        p.ref.pool[page, 0, which, 0, t % 16, 3] = x
    q, out, ref, slots, sc = attend(p, [rows], 2, window=rows // 2, sinks=2)
    o = np64(out)
    odd = ~np.isfinite(ref)
    assert odd.any() and not odd.all()
    assert not np.isfinite(o[odd]).any()
    if which == 1:
        assert np.array_equal(np.isnan(o), np.isnan(ref))
        inf = np.isinf(ref)
        assert np.array_equal(o[inf], ref[inf])
    fine = np.isfinite(ref).all(axis=(1, 2))
    assert fine.any()
    ok = torch.from_numpy(np.where(np.isfinite(ref), o, 0))
    check_out(ok, np.where(np.isfinite(ref), ref, 0), dtype, q, p, 0, slots, [rows], sc)


def test_scores_of_minus_infinity_are_not_an_empty_row():
    """A row whose every visible score is -inf has no softmax: NaN, not 0."""
    p = Pair([20], "f16", 16, 1, 64)
    p.gpu.pool[:, 0, 0] = 0
    p.gpu.pool[:, 0, 0, :, :, 0] = float("-inf")
    for rows in (1, 20):
        q = torch.zeros((rows, 8, 64), dtype=torch.float16, device="cuda")
        q[:, :, 0] = 1
        assert torch.isnan(p.gpu.attend(q, seqs=[0])).all()


def test_large_scores_do_not_overflow():
    p = Pair([100], "f16", 16, 1, 128)
    p.gpu.pool[:, 0, 0] *= 100
    p.ref.pool[:, 0, 0] = np64(p.gpu.pool[:, 0, 0])
    q, out, ref, slots, sc = attend(p, [1], 4, scale=1.0)
    o = np64(out)
    assert np.isfinite(o).all()
    # one token takes nearly all the weight
    assert np.abs(o - ref).max() <= 0.05


@pytest.mark.parametrize("rows", [1, 8, 120])
def test_strides_and_layers(rows):
    """q as columns of stacked q|k|v rows, out as columns of a wider tensor, a layer in the middle."""
    p = Pair([rows + 40, rows + 3], "f16", 16, 2, 64, layers=3)
    q = rand((2 * rows, 4, 64), "f16", 3)
    wide = torch.zeros((2 * rows, 12, 64), dtype=torch.float16, device="cuda")
    wide[:, 2:6] = q
    res = torch.full((2 * rows, 9, 64), 7.0, dtype=torch.float16, device="cuda")
    out = p.gpu.attend(wide[:, 2:6], layer=1, out=res[:, 4:8], seqs=[0, 1])
    assert out.data_ptr() == res[:, 4:8].data_ptr()
    ref = p.ref.attend(1, [0, 1], [rows] * 2, np64(q), 0.125)
    check_out(out, ref, "f16", q, p, 1, [0, 1], [rows] * 2, 0.125)
    assert (res[:, :4] == 7).all() and (res[:, 8:] == 7).all()


@pytest.mark.parametrize("rows", [1, 8, 120])
def test_bits_repeat(rows):
    p = Pair([700, 3, 1200, rows + 9], "bf16", 16, 4, 128)
    q = rand((4 * rows, 8, 128), "bf16", 4)
    first = p.gpu.attend(q, seqs=[0, 1, 2, 3])
    for _ in range(3):
        assert torch.equal(first.view(torch.int16), p.gpu.attend(q, seqs=[0, 1, 2, 3]).view(torch.int16))


def test_another_stream():
    p = Pair([300, 40], "f16", 16, 2, 128)
    q = rand((2, 8, 128), "f16", 4)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    a = p.gpu.attend(q, seqs=[0, 1], stream=s)
    s.synchronize()
    assert torch.equal(a, p.gpu.attend(q, seqs=[0, 1]))


def test_many_slots():
    """More entries than lanes of a wave, in an order of their own, one named out of range (it acts as empty)."""
    n = 150
    lens = [1 + (37 * i) % 90 for i in range(n)]
    p = Pair(lens, "f16", 16, 1, 64)
    slots = list(np.random.default_rng(0).permutation(n))
    out = run(p, [1] * n, 3, slots=[int(s) for s in slots], uniform=True)
    assert out.shape == (n, 3, 64)
    q = rand((2, 3, 64), "f16", 4)
    o = p.gpu.attend(q, seqs=[5, n + 7])
    assert (o[1] == 0).all() and (o[0] != 0).any()


def test_table_ids_out_of_range_stay_in_the_pool():
    """A page id that names no page is read as page 0: no fault, and a defined result."""
    p = Pair([100], "f16", 16, 1, 64)
    p.gpu.tables[0, 2] = 1 << 30
    p.gpu.tables[0, 3] = -5
    p.ref.tables[0, 2] = 0
    p.ref.tables[0, 3] = 0
    run(p, [1], 2)
    run(p, [70], 2)


def test_lengths_out_of_range_are_cut():
    p = Pair([64], "f16", 16, 1, 64, max_pages=4)
    q = rand((1, 2, 64), "f16", 4)
    a = p.gpu.attend(q, seqs=[0])
    p.gpu.lens.fill_(1 << 30)
    assert torch.equal(a, p.gpu.attend(q, seqs=[0]))
    p.gpu.lens.fill_(-3)
    assert (p.gpu.attend(q, seqs=[0]) == 0).all()


def test_graph_replay_follows_lengths_and_tables():
    """A captured append + attend reads lens, tables and rows at each replay."""
    p = Pair([40, 9], "f16", 16, 2, 128, extra=8, max_pages=8)
    q, k, v = (rand((2, h, 128), "f16", 5 + h) for h in (10, 2, 2))
    v = rand((2, 2, 128), "f16", 11)
    one = torch.ones(2, dtype=torch.int32, device="cuda")
    seqs = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    out = torch.empty_like(q)

    def step():
        p.gpu.extend(one)
        p.gpu.append(k, v, seqs=seqs)
        p.gpu.attend(q, seqs=seqs, out=out)

    step()
    p.ref.extend([1, 1])
    p.ref.append(0, [0, 1], [1, 1], np64(k), np64(v))
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for i in range(5):
        q.copy_(rand(q.shape, "f16", 100 + i))
        k.copy_(rand(k.shape, "f16", 200 + i))
        g.replay()
        torch.cuda.synchronize()
        p.ref.extend([1, 1])
        p.ref.append(0, [0, 1], [1, 1], np64(k), np64(v))
        p.same_state()
        check_out(out, p.ref.attend(0, [0, 1], [1, 1], np64(q), 128 ** -0.5), "f16", q, p, 0, [0, 1], [1, 1], 128 ** -0.5)


def test_refusals():
    p = Pair([40, 9], "f16", 16, 2, 64, layers=2)
    kv = p.gpu
    q = rand((2, 4, 64), "f16", 4)
    for bad in (dict(layer=2), dict(layer=-1), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")),
                dict(window=-1), dict(sinks=-1), dict(seqs=[0, 1, 1]), dict(row_start=[0, 1, 2], max_rows=0),
                dict(row_start=[0, 1, 2], max_rows=3)):
        with pytest.raises(Q.QGError):
            kv.attend(q, **{"seqs": [0, 1], **bad})
    for bad in (q[:, :3], q[:1].expand(3, 4, 64)):
        with pytest.raises(Q.QGError):
            kv.attend(bad, seqs=[0, 1])
    for bad in (q.float(), q.bfloat16(), q[:, :, :32], q[0], q.transpose(1, 2), q.cpu()):
        with pytest.raises((ValueError, Q.QGError)):
            kv.attend(bad, seqs=[0, 1])
    with pytest.raises(ValueError):
        kv.attend(q, row_start=[0, 1, 2])
    with pytest.raises(ValueError):
        kv.attend(q, seqs=torch.tensor([0, 1], device="cuda"))
    odd = torch.zeros(2 * 4 * 64 + 8, dtype=torch.float16, device="cuda")
    with pytest.raises(Q.QGError, match="aligned"):
        kv.attend(odd[1:1 + 512].view(2, 4, 64), seqs=[0, 1])
    with pytest.raises(Q.QGError, match="strides"):
        kv.attend(torch.zeros((2, 4 * 64 + 4), dtype=torch.float16, device="cuda")[:, :256].view(2, 4, 64), seqs=[0, 1])
    kv.close()
    with pytest.raises(ValueError, match="closed"):
        kv.attend(q)
