"""Rotary positions alone and on the way into the cache, against their definition in fp64."""
from __future__ import annotations

import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from _kv import DT, UNIT, Pair, np64, rand  # noqa: E402
from oracle import step_oracle as SO  # noqa: E402
import bit_weight_only_packed_amd as Q  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _gpu_present():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def check(out, x, ref, dtype, dim, size=1.0):
    """Angles to 2 pi (2^-25 + 2^-33) turns (the fraction's rounding to 24 bits), sines to 2^-22, three fp32 roundings:
    2^-21 of |a| + |b| covers them; and the output's rounding.  What is not rotated is the same."""
    big = np.abs(np64(x)).max(-1, keepdims=True) * 2 * max(abs(size), 1e-30)
    err = np.abs(np64(out) - ref)
    tol = UNIT[dtype] * np.abs(ref) + 2.0 ** -21 * big + 2.0 ** -25
    assert (err <= tol)[..., :dim].all(), float((err / tol)[..., :dim].max())
    assert torch.equal(out[..., dim:], x[..., dim:])


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("rows,heads,d,dim", [(1, 1, 16, 16), (3, 5, 64, 64), (7, 2, 80, 48), (2, 40, 128, 128), (5, 3, 128, 32),
                                              (300, 8, 128, 128), (33, 1, 256, 64), (2, 2, 1024, 1024), (2100, 3, 64, 16)])
def test_against_the_definition(dtype, pairs, rows, heads, d, dim):
    r = Q.Rotary(dim, 10000.0, interleaved=pairs)
    x = rand((rows, heads, d), dtype, rows + d)
    pos = torch.from_numpy(np.random.default_rng(rows).integers(0, 9000, rows).astype(np.int32)).cuda()
    out = r.rotate(x, pos)
    check(out, x, SO.rotate(np64(x), pos.tolist(), r.freqs, 1.0, pairs), dtype, dim)
    back = r.rotate(x, pos, out=x.clone())
    assert torch.equal(back, out)
    y = x.clone()
    assert r.rotate(y, pos, out=y).data_ptr() == y.data_ptr() and torch.equal(y, out)  # in place


@pytest.mark.parametrize("scaling", ["linear", "ntk", "yarn"])
def test_scalings_far_along(scaling):
    """Positions up to 2^24: the oracle's own angle is off by 2^-53 of itself, 2^-29."""
    r = Q.Rotary(64, 500000.0, scaling=scaling, factor=8.0, original=8192)
    x = rand((9, 2, 128), "f16", 5)
    pos = [0, 1, 4095, 8191, 65537, 1 << 20, (1 << 20) + 1, (1 << 24) - 1, 1 << 24]
    out = r.rotate(x, torch.tensor(pos, dtype=torch.int32, device="cuda"))
    check(out, x, SO.rotate(np64(x), pos, r.freqs, r.size), "f16", 64, r.size)


def test_any_position():
    """Frequencies of whole 64ths of a turn: the angle at any position is one of 64, also at the ends of int32."""
    k = np.arange(16) * 5 + 1
    r = Q.Rotary.of(2 * math.pi * k / 64, size=0.5, interleaved=True)
    pos = np.array([2 ** 31 - 1, -2 ** 31, -1, 2 ** 30 + 7, 12345678, 0], dtype=np.int64)
    x = rand((6, 3, 32), "bf16", 6)
    out = r.rotate(x, torch.from_numpy(pos.astype(np.int32)).cuda())
    small = [int(p) % 64 for p in pos]
    check(out, x, SO.rotate(np64(x), small, r.freqs, 0.5, True), "bf16", 32, 0.5)


def test_strided_rows_and_columns():
    """q in the columns of stacked rows, rotated in place: the other columns stay."""
    t = rand((11, 12, 64), "f16", 7)
    keep, pos = t.clone(), torch.arange(11, dtype=torch.int32, device="cuda") * 3
    r = Q.Rotary(64)
    r.rotate(t[:, 2:9], pos, out=t[:, 2:9])
    assert torch.equal(t[:, :2], keep[:, :2]) and torch.equal(t[:, 9:], keep[:, 9:])
    check(t[:, 2:9], keep[:, 2:9], SO.rotate(np64(keep[:, 2:9]), pos.tolist(), r.freqs), "f16", 64)
    # heads slowest
    h = rand((4, 11, 64), "f16", 8)
    out = torch.empty_like(h)
    r.rotate(h.transpose(0, 1), pos, out=out.transpose(0, 1))
    check(out.transpose(0, 1), h.transpose(0, 1), SO.rotate(np64(h.transpose(0, 1)), pos.tolist(), r.freqs), "f16", 64)
    # out in other columns of x's rows
    r.rotate(t[:, :4], pos, out=t[:, 4:8])
    check(t[:, 4:8], t[:, :4], SO.rotate(np64(t[:, :4]), pos.tolist(), r.freqs), "f16", 64)


def test_refusals():
    r = Q.Rotary(64)
    x, pos = rand((4, 2, 64), "f16", 1), torch.zeros(4, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="positions"):
        r.rotate(x, pos.long())
    with pytest.raises(ValueError, match="positions"):
        r.rotate(x, pos[:3])
    with pytest.raises(ValueError, match="float16"):
        r.rotate(x.float(), pos)
    with pytest.raises(ValueError, match="out"):
        r.rotate(x, pos, out=x[:, :1])
    with pytest.raises(Q.QGError, match="dim"):
        r.rotate(x[..., :32], pos)
    with pytest.raises(Q.QGError, match="overlaps"):
        r.rotate(x[:3], pos[:3], out=x[1:])
    assert r.rotate(x[:0], pos[:0]).shape == (0, 2, 64)


# ------------------------------------------------------------------------------------------------- into the cache

def written(pair, slots, rows, k, v, rot, layer=0):
    """The oracle's cache after the rows: k rotated in fp64, rounded by torch."""
    at = 0
    for s, n in zip(slots, rows):
        for i in range(n):
            pos = int(pair.ref.lens[s]) - n + i
            if pos >= 0:
                kk = SO.rotate(np64(k[at + i:at + i + 1]), [pos], rot.freqs, rot.size, rot.interleaved)[0]
                page, slot = int(pair.ref.tables[s, pos // pair.ref.P]), pos % pair.ref.P
                pair.ref.pool[page, layer, 0, :, slot], pair.ref.pool[page, layer, 1, :, slot] = kk, np64(v[at + i])
        at += n


def same_pool(pair, k, dtype):
    """Keys to their rounding, everything else bit for bit."""
    torch.cuda.synchronize()
    got, want = np64(pair.gpu.pool), pair.ref.pool
    big = float(np.abs(np64(k)).max()) * 4
    assert np.array_equal(got[:, :, 1], want[:, :, 1])
    assert (np.abs(got - want) <= UNIT[dtype] * np.abs(want) + 2.0 ** -21 * big + 2.0 ** -25).all()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("D,heads,qh,page,dim,pairs", [(64, 2, 6, 16, 64, False), (128, 1, 8, 32, 64, True), (256, 3, 3, 16, 256, False),
                                                       (128, 8, 40, 64, 128, True)])
def test_append(dtype, D, heads, qh, page, dim, pairs):
    lens, rows = [5, 37, 0, 130, 16, 64], [5, 3, 1, 33, 0, 1]
    pair = Pair(lens, dtype, page, heads, D, layers=2, seed=D + page)
    rot = Q.Rotary(dim, 1000.0, interleaved=pairs, scaling="yarn", factor=3.0, original=64)
    n = sum(rows)
    qkv = rand((n, qh + 2 * heads, D), dtype, 3)
    q, k, v = qkv.split([qh, heads, heads], 1)
    start = torch.tensor([0] + list(np.cumsum(rows)), dtype=torch.int32, device="cuda")
    seqs = torch.tensor([3, 0, 2, 1, 4, 5], dtype=torch.int32, device="cuda")
    order, count = seqs.tolist(), rows
    out = pair.gpu.append_rotated(q, k, v, rot, layer=1, seqs=seqs, row_start=start, max_rows=33)
    before = pair.ref.pool.copy()
    written(pair, order, count, k, v, rot, 1)
    same_pool(pair, k, dtype)
    assert np.array_equal(np64(pair.gpu.pool[:, 0]), before[:, 0])
    at = 0
    for s, r in zip(order, count):
        pos = [lens[s] - r + i for i in range(r)]
        live = [i for i in range(r) if pos[i] >= 0]
        if live:
            part = slice(at + live[0], at + r)
            check(out[part], q[part], SO.rotate(np64(q[part]), [pos[i] for i in live], rot.freqs, rot.size, pairs), dtype, dim, rot.size)
        assert (out[at:at + r - len(live)] == 0).all()
        at += r
    # in place over the columns of q, and keys alone: the same pages
    want, pool = out.clone(), pair.gpu.pool.clone()
    pair.gpu.pool[:, 1].zero_()
    assert pair.gpu.append_rotated(None, k, v, rot, layer=1, seqs=seqs, row_start=start, max_rows=33) is None
    again = pair.gpu.pool.clone()
    pair.gpu.pool[:, 1].zero_()
    pair.gpu.append_rotated(q, k, v, rot, layer=1, seqs=seqs, row_start=start, max_rows=33, out=q)
    torch.cuda.synchronize()
    assert torch.equal(q, want) and torch.equal(pair.gpu.pool, again)
    rows_written = (again[:, 1] != 0).any(-1)
    assert torch.equal(again[:, 1][rows_written], pool[:, 1][rows_written])


def test_left_out_rows_keep_their_output():
    """Rows past max_rows and behind the last entry."""
    pair = Pair([40, 40], "f16", 16, 1, 64, seed=4)
    k, q = rand((12, 1, 64), "f16", 1), rand((12, 2, 64), "f16", 2)
    rot = Q.Rotary(64)
    out = torch.full_like(q, 9.0)
    start = torch.tensor([0, 6, 8], dtype=torch.int32, device="cuda")
    pair.gpu.append_rotated(q, k, k, rot, row_start=start, max_rows=4, out=out)
    torch.cuda.synchronize()
    assert (out[4:6] == 9).all() and (out[8:] == 9).all()
    for rows, pos in ((slice(0, 4), range(34, 38)), (slice(6, 8), range(38, 40))):
        check(out[rows], q[rows], SO.rotate(np64(q[rows]), list(pos), rot.freqs), "f16", 64)


def test_equals_rotate_then_append():
    """Bit for bit what the two calls give that it stands for."""
    pair, other = (Pair([70, 9, 200], "bf16", 32, 2, 128, seed=9) for _ in range(2))
    q, k, v = rand((6, 4, 128), "bf16", 1), rand((6, 2, 128), "bf16", 2), rand((6, 2, 128), "bf16", 3)
    rot = Q.Rotary(128, interleaved=True)
    out = pair.gpu.append_rotated(q, k, v, rot, seqs=[0, 1, 2])
    pos = torch.tensor([68, 69, 7, 8, 198, 199], dtype=torch.int32, device="cuda")
    other.gpu.append(rot.rotate(k, pos), v, seqs=[0, 1, 2])
    torch.cuda.synchronize()
    assert torch.equal(out, rot.rotate(q, pos)) and torch.equal(pair.gpu.pool, other.gpu.pool)


def test_nothing_is_written_while_a_refused_extend_stands():
    pair = Pair([16, 16], "f16", 16, 1, 64, extra=0, max_pages=4)
    keep = pair.gpu.pool.clone()
    pair.gpu.extend([100, 0])
    q, k = rand((2, 1, 64), "f16", 1), rand((2, 1, 64), "f16", 2)
    out = pair.gpu.append_rotated(q, k, k, Q.Rotary(64))
    torch.cuda.synchronize()
    assert torch.equal(pair.gpu.pool, keep)
    check(out, q, SO.rotate(np64(q), [15, 15], Q.Rotary(64).freqs), "f16", 64)
    with pytest.raises(Q.QGError):
        pair.gpu.check()


def test_bad_pages_are_not_written():
    """Page ids out of the pool, slots out of range: nothing is written through them, and q is rotated as ever."""
    pair = Pair([20, 20], "f16", 16, 1, 64, seed=2)
    pair.gpu.tables[0, 1], pair.gpu.tables[1, 1] = 1 << 20, -5
    keep = pair.gpu.pool.clone()
    q, k = rand((3, 1, 64), "f16", 1), rand((3, 1, 64), "f16", 2)
    rot = Q.Rotary(64)
    out = pair.gpu.append_rotated(q[:2], k[:2], k[:2], rot)
    torch.cuda.synchronize()
    assert torch.equal(pair.gpu.pool, keep)
    check(out, q[:2], SO.rotate(np64(q[:2]), [19, 19], rot.freqs), "f16", 64)
    out = pair.gpu.append_rotated(q[:1], k[:1], k[:1], rot, seqs=[7])
    torch.cuda.synchronize()
    assert torch.equal(pair.gpu.pool, keep) and (out == 0).all()


def test_append_refusals():
    pair = Pair([20], "f16", 16, 2, 64)
    kv, rot = pair.gpu, Q.Rotary(64)
    q, k = rand((4, 2, 64), "f16", 1), rand((4, 2, 64), "f16", 2)
    with pytest.raises(ValueError, match="q must"):
        kv.append_rotated(q[:3], k, k, rot, seqs=[0])
    with pytest.raises(ValueError, match="out without q"):
        kv.append_rotated(None, k, k, rot, seqs=[0], out=q)
    with pytest.raises(Q.QGError, match="dim"):
        kv.append_rotated(q, k, k, Q.Rotary(128), seqs=[0])
    with pytest.raises(Q.QGError, match="overlaps k or v"):
        kv.append_rotated(q, k, k, rot, seqs=[0], out=k)
    with pytest.raises(Q.QGError, match="overlaps q"):
        kv.append_rotated(q[:3], k[:3], k[:3], rot, seqs=[0], out=q[1:])
    with pytest.raises(Q.QGError, match="layer"):
        kv.append_rotated(q, k, k, rot, seqs=[0], layer=1)


def test_a_captured_step():
    """Replays follow lengths that grow, as eager calls do."""
    kvs = [Q.KVCache(16, 16, 2, 64, max_seqs=3, max_pages=5) for _ in range(2)]
    rot = Q.Rotary(64)
    grow = torch.tensor([1, 0, 2], dtype=torch.int32, device="cuda")
    start = torch.tensor([0, 1, 1, 3], dtype=torch.int32, device="cuda")
    qkv = rand((3, 8, 64), "f16", 5)
    q, k, v = qkv.split([4, 2, 2], 1)
    out = torch.empty((3, 4, 64), dtype=torch.float16, device="cuda")
    for kv in kvs:
        kv.pool.zero_()
        kv.extend([7, 1, 0])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kvs[0].extend(grow)
        kvs[0].append_rotated(q, k, v, rot, row_start=start, max_rows=2, out=out)
    for i in range(6):
        qkv.copy_(rand((3, 8, 64), "f16", 10 + i))
        graph.replay()
        kvs[1].extend(grow)
        want = kvs[1].append_rotated(q, k, v, rot, row_start=start, max_rows=2)
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(kvs[0].pool, kvs[1].pool)
        assert torch.equal(kvs[0].lens, kvs[1].lens)
