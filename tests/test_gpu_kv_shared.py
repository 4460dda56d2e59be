"""Attention of entries that share their first pages: against the oracle, which attends to each by itself."""
from __future__ import annotations

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from _kv import Pair, check_out, np64, rand  # noqa: E402
from oracle import kv_oracle as KO  # noqa: E402
import bit_weight_only_packed_amd as Q  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _gpu_present():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


class Always(Q.KVCache):
    """A cache whose attend_shared shares whatever entries have in common, also where that does not pay."""

    def attend_shared(self, q, **kw):
        return super().attend_shared(q, **{"least": 0, **kw})


class Forked(Pair):
    """Prompts of given lengths, each forked to slots that then grow by their own tokens.
    answers: for each prompt the tokens that its slots add; slots in order, the prompts' own slots last."""

    def __init__(self, prompts, answers, dtype="f16", page=16, heads=2, D=64, seed=1, fill=None):
        n = sum(map(len, answers))
        room = sum(-(-(p + x) // page) + 1 for p, a in zip(prompts, answers) for x in a)
        longest = max(p + max(a) for p, a in zip(prompts, answers))
        super().__init__([0] * n + list(prompts), dtype, page, heads, D, extra=room, max_pages=-(-longest // page) + 2, seed=seed,
                         fill=fill)
        g = self.gpu
        self.gpu = Always.of(g.pool, g.tables, g.lens, g.refs)
        kv, at = self.gpu, 0
        grow = torch.zeros(kv.max_seqs, dtype=torch.int32)
        for i, a in enumerate(answers):
            kv.fork([n + i] * len(a), list(range(at, at + len(a))))
            grow[at:at + len(a)] = torch.tensor(a, dtype=torch.int32)
            at += len(a)
        kv.extend(grow.cuda())
        # the tokens that were added hold values, and the copied tails' rest what `fill` says
        lens = kv.lens.cpu().numpy()
        for s in range(n):
            for t in range(int(lens[s]) - int(grow[s]), int(lens[s])):
                p = int(kv.tables[s, t // page])
                kv.pool[p, :, :, :, t % page] = rand((kv.layers, 2, heads, D), dtype, 1000 * s + t)
        kv.check()
        self.again()

    def again(self):
        kv = self.gpu
        torch.cuda.synchronize()
        self.ref = KO.Cache(np64(kv.pool), kv.tables.cpu().numpy(), kv.lens.cpu().numpy(), kv.refs.cpu().numpy())

    def check(self, q, out, slots, rows, window=0, sinks=0, dtype="f16", scale=None):
        scale = self.gpu.head_dim ** -0.5 if scale is None else scale
        ref = self.ref.attend(0, slots, rows, np64(q), scale, window, sinks)
        check_out(out, ref, dtype, q, self, 0, slots, rows, scale)


def ints(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("D,heads,G,page", [(64, 2, 4, 16), (128, 2, 5, 32), (256, 1, 8, 16), (128, 1, 1, 64), (64, 1, 16, 256)])
@pytest.mark.parametrize("prompt,own", [(300, [1, 5, 40, 17]), (1027, [3, 70]), (512, [1, 1, 64, 200, 9, 30, 2])])
def test_one_token_each(dtype, D, heads, G, page, prompt, own):
    f = Forked([prompt], [own], dtype, page, heads, D, seed=D + prompt)
    q = rand((len(own), heads * G, D), dtype, 3, 1.5)
    slots = list(range(len(own)))
    out = f.gpu.attend_shared(q, seqs=ints(*slots))
    f.check(q, out, slots, [1] * len(own), dtype=dtype)
    assert torch.equal(f.gpu.attend_shared(q), out)  # the same bits again, and slots by default


@pytest.mark.parametrize("dtype,D,heads,G", [("f16", 128, 2, 5), ("bf16", 256, 2, 4), ("f16", 64, 1, 8), ("bf16", 128, 1, 40)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (100, 0), (700, 5), (1, 0), (513, 70), (100000, 3)])
def test_verify_rows_groups_and_windows(dtype, D, heads, G, window, sinks):
    """Two groups of ragged rows, an idle entry, an entry without rows; both kernels for the entries' own tokens."""
    f = Forked([900, 520], [[9, 30, 4], [6, 100, 8, 1]], dtype, 16, heads, D, seed=5)
    f.gpu.trim(ints(1))  # idle
    f.again()
    slots, rows = [2, 1, 0, 3, 4, 6, 5], [3, 1, 5, 6, 0, 1, 4]
    start = ints(0, *np.cumsum(rows).tolist())
    q = rand((sum(rows), heads * G, D), dtype, 4, 1.5)
    kw = dict(seqs=ints(*slots), row_start=start, max_rows=6, window=window, sinks=sinks)
    out = f.gpu.attend_shared(q, groups=ints(0, 3, 7), **kw)
    f.check(q, out, slots, rows, window, sinks, dtype)
    # entries of both prompts in one group share nothing; every entry for itself neither
    for groups in (None, ints(0, 7), ints(*range(8))):
        f.check(q, f.gpu.attend_shared(q, groups=groups, **kw), slots, rows, window, sinks, dtype)


def test_long_prompt_in_many_parts():
    f = Forked([9000], [[3, 50, 7, 12, 100, 1, 2, 8]], "bf16", 64, 2, 128, seed=7)
    q = rand((8, 10, 128), "bf16", 5, 1.5)
    f.check(q, f.gpu.attend_shared(q), list(range(8)), [1] * 8, dtype="bf16")


def test_more_rows_than_a_block():
    """Rows of one entry on both sides of a block's edge."""
    f = Forked([700], [[9 + i for i in range(17)]], "f16", 16, 2, 64, seed=8)
    rows = [1 + i % 4 for i in range(17)]
    start = ints(0, *np.cumsum(rows).tolist())
    q = rand((sum(rows), 14, 64), "f16", 6, 1.5)
    out = f.gpu.attend_shared(q, seqs=ints(*range(17)), row_start=start, max_rows=4)
    f.check(q, out, list(range(17)), rows)


def test_rows_that_the_shared_tokens_hold():
    """Verify rows that lie inside the shared pages: what is shared ends before the first of them."""
    f = Forked([800], [[1, 2, 30]], "f16", 16, 1, 128, seed=9)
    rows = [300, 7, 40]
    start = ints(0, *np.cumsum(rows).tolist())
    q = rand((sum(rows), 2, 128), "f16", 6, 1.5)
    out = f.gpu.attend_shared(q, seqs=ints(0, 1, 2), row_start=start, max_rows=300)
    f.check(q, out, [0, 1, 2], rows)


def test_entries_that_are_one_slot():
    """The same slot twice, and a prompt's own slot beside its forks."""
    f = Forked([640], [[2, 9, 5]], "f16", 16, 1, 64, seed=10)
    slots = [0, 1, 0, 3]
    q = rand((4, 4, 64), "f16", 7, 1.5)
    f.check(q, f.gpu.attend_shared(q, seqs=ints(*slots)), slots, [1] * 4)
    f.check(q[:2], f.gpu.attend_shared(q[:2], seqs=ints(2, 2)), [2, 2], [1, 1])


def test_only_idle_entries_and_single_ones():
    f = Forked([640], [[2, 9, 4]], "f16", 16, 1, 64, seed=11)
    q = rand((3, 4, 64), "f16", 8, 1.5)
    f.check(q[:1], f.gpu.attend_shared(q[:1], seqs=ints(1)), [1], [1])
    f.gpu.trim(ints(0, 2))
    f.again()
    f.check(q, f.gpu.attend_shared(q, seqs=ints(0, 1, 2)), [0, 1, 2], [1] * 3)
    f.gpu.trim(ints(1))
    assert (f.gpu.attend_shared(q, seqs=ints(0, 1, 2)) == 0).all()
    assert f.gpu.attend_shared(q[:0]).shape == (0, 4, 64)


def test_memory_that_no_row_sees_never_reaches_one():
    """NaN in all memory that holds no token, and tokens outside the window."""
    f = Forked([700], [[1, 40, 18]], "f16", 64, 2, 64, seed=12, fill=float("nan"))
    q = rand((3, 6, 64), "f16", 9, 1.5)
    for window, sinks in ((0, 0), (200, 3)):
        out = f.gpu.attend_shared(q, window=window, sinks=sinks)
        assert torch.isfinite(out).all()
        f.check(q, out, [0, 1, 2], [1] * 3, window, sinks)


def test_non_finite_tokens_reach_the_rows_that_see_them():
    f = Forked([700], [[1, 300]], "bf16", 16, 1, 64, seed=13)
    page = int(f.gpu.tables[0, 390 // 16])
    f.gpu.pool[page, 0, 1, 0, 390 % 16, 5] = float("inf")  # token 390: slot 0 sees it through the window, slot 1 not
    f.again()
    q = rand((2, 3, 64), "bf16", 9, 1.5)
    out = f.gpu.attend_shared(q, window=400)
    assert torch.isinf(out[0, :, 5]).all() and torch.isfinite(out[1]).all()
    keep = torch.arange(64, device="cuda") != 5
    assert torch.isfinite(out[0][:, keep]).all()
    out = f.gpu.attend_shared(q)
    assert torch.isinf(out[:, :, 5]).all()


def test_weights_far_below_the_largest():
    """Shared tokens of scores far below the own ones', and the other way round: both sides' exponents mean the same."""
    for dtype in ("f16", "bf16"):
        for own_scale, prompt_scale in ((3.0, 0.1), (0.1, 3.0)):
            f = Forked([512], [[20, 33]], dtype, 16, 1, 64, seed=14)
            kv = f.gpu
            for s in range(2):
                for i in range(int(kv.lens[s] + 15) // 16):
                    kv.pool[int(kv.tables[s, i]), 0, 0] = rand((1, 16, 64), dtype, i, prompt_scale if i < 32 else own_scale)
            f.again()
            q = rand((2, 4, 64), dtype, 10, 2.0)
            f.check(q, kv.attend_shared(q), [0, 1], [1, 1], dtype=dtype)


def test_tables_and_groups_that_make_no_sense():
    """Ids out of the pool, slots out of range, groups that descend, overlap or leave the call: nothing leaves memory,
    and entries that are in order come out right."""
    f = Forked([600, 600], [[5, 9, 17], [3, 8]], "f16", 16, 1, 64, seed=15)
    q = rand((5, 4, 64), "f16", 11, 1.5)
    want = f.gpu.attend_shared(q, groups=ints(0, 3, 5))
    f.check(q, want, list(range(5)), [1] * 5)
    out = f.gpu.attend_shared(q, seqs=ints(0, 99, 2, -1, 4), groups=ints(0, 3, 5))
    assert (out[[1, 3]] == 0).all()
    f.check(out=out[[0, 2, 4]], q=q[[0, 2, 4]], slots=[0, 2, 4], rows=[1] * 3)
    for groups in (ints(3, 0, 5), ints(-7, 100, 3), ints(5, 5, 5), ints(0, 1 << 30, -(1 << 30)), ints(0, 4, 2, 5)):
        out = f.gpu.attend_shared(q, groups=groups)
        f.check(q, out, list(range(5)), [1] * 5)
    f.gpu.tables[0, 3], f.gpu.tables[1, 3] = 1 << 30, 1 << 30  # read as page 0, by both
    f.gpu.tables[2, 3] = -4
    out = f.gpu.attend_shared(q, groups=ints(0, 3, 5))
    tables = f.ref.tables.copy()
    f.ref.tables[:3, 3] = 0
    f.check(q, out, list(range(5)), [1] * 5)
    f.ref.tables = tables


def test_left_out_rows_and_rows_behind_the_last():
    f = Forked([600], [[30, 40]], "f16", 16, 1, 64, seed=16)
    q = rand((14, 4, 64), "f16", 12, 1.5)
    out = torch.full_like(q, 5.0)
    f.gpu.attend_shared(q, row_start=ints(0, 7, 12), max_rows=3, out=out, window=20)
    assert (out[3:7] == 5).all() and (out[10:] == 5).all()
    ref = f.ref.attend(0, [0, 1], [7, 5], np64(q[:12]), 0.125, 20, 0)
    for a in (0, 7):
        assert np.abs(np64(out[a:a + 3]) - ref[a:a + 3]).max() < 2e-3 * np.abs(ref).max()


def test_calls_of_very_many_rows():
    """More rows than the workspace has slots for go the usual way."""
    f = Forked([320], [[40] * 2], "f16", 16, 8, 64, seed=17)
    q = rand((2 * 1100, 64, 64), "f16", 13, 1.5)
    small = dict(seqs=ints(0, 1), row_start=ints(0, 2199, 2200), max_rows=2199)
    a, b = f.gpu.attend_shared(q, **small), f.gpu.attend(q, **small)
    assert torch.equal(a, b)


def test_where_it_does_not_pay():
    """Below `least` the call is attend, bit for bit: by the slots' room on the host, by the shared tokens on the device."""
    f = Forked([1000], [[3, 40, 20]], "f16", 16, 2, 64, seed=20)
    q = rand((3, 8, 64), "f16", 16, 1.5)
    plain, shared = f.gpu.attend(q), f.gpu.attend_shared(q)
    f.check(q, shared, [0, 1, 2], [1] * 3)
    token = 2 * 2 * 64 * 2
    assert torch.equal(f.gpu.attend_shared(q, least=-1), plain)
    assert torch.equal(f.gpu.attend_shared(q, least=3 * f.gpu.max_pages * 16 * token + token), plain)
    assert torch.equal(f.gpu.attend_shared(q, least=3 * 960 * token), shared)          # 960 of the 1,000 are shared
    assert torch.equal(f.gpu.attend_shared(q, least=3 * 960 * token + token), plain)
    # a group that shares little comes along with one that shares enough
    two = Forked([1000, 300], [[3, 40], [5, 6]], "f16", 16, 2, 64, seed=21)
    q = rand((4, 8, 64), "f16", 17, 1.5)
    both = two.gpu.attend_shared(q, groups=ints(0, 2, 4))
    assert torch.equal(two.gpu.attend_shared(q, groups=ints(0, 2, 4), least=2 * (960 + 256) * token), both)
    assert torch.equal(two.gpu.attend_shared(q, groups=ints(0, 2, 4), least=2 * (960 + 256) * token + token), two.gpu.attend(q))


def test_strided_operands_and_refusals():
    f = Forked([600], [[3, 4]], "f16", 16, 2, 64, seed=18)
    qkv, out = rand((2, 12, 64), "f16", 14, 1.5), torch.zeros((8, 2, 64), dtype=torch.float16, device="cuda")
    q = qkv[:, 2:10]
    got = f.gpu.attend_shared(q, out=out.transpose(0, 1))
    f.check(q, got, [0, 1], [1, 1])
    with pytest.raises(Q.QGError, match="n_groups"):
        f.gpu.attend_shared(q, groups=ints(0, 1, 2, 2))
    with pytest.raises(Q.QGError, match="n_groups"):
        f.gpu.attend_shared(q, groups=ints(0))
    with pytest.raises(ValueError, match="groups"):
        f.gpu.attend_shared(q, groups=torch.zeros(2, dtype=torch.int64, device="cuda"))
    with pytest.raises(Q.QGError, match="overlaps q"):
        f.gpu.attend_shared(q, out=q)
    with pytest.raises(Q.QGError, match="q_heads"):
        f.gpu.attend_shared(qkv[:, :3])
    with pytest.raises(Q.QGError, match="scale"):
        f.gpu.attend_shared(q, scale=-1.0)


def test_other_streams_and_calls_between():
    f = Forked([2000], [[3, 4, 90]], "f16", 16, 2, 64, seed=19)
    q = rand((3, 8, 64), "f16", 15, 1.5)
    want, plain = f.gpu.attend_shared(q), f.gpu.attend(q)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = f.gpu.attend_shared(q, stream=side)
    other = f.gpu.attend(q, stream=side)
    again = f.gpu.attend_shared(q, stream=side)
    side.synchronize()
    assert torch.equal(got, want) and torch.equal(again, want) and torch.equal(other, plain)


def test_a_captured_step_follows_the_tables():
    """Replays after forks, trims and growth give what eager calls give: what is shared is found anew each time."""
    kv = Always(200, 16, 2, 64, max_seqs=4, max_pages=60)
    kv.extend([600, 0, 0, 0])
    kv.append(rand((600, 2, 64), "f16", 1), rand((600, 2, 64), "f16", 2), seqs=[0])
    kv.fork([0, 0, 0], [1, 2, 3])
    grow, q = ints(1, 1, 1, 1), rand((4, 8, 64), "f16", 3, 1.5)
    k, v = rand((4, 2, 64), "f16", 4), rand((4, 2, 64), "f16", 5)
    out = torch.empty_like(q)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kv.extend(grow)
        kv.append(k, v)
        kv.attend_shared(q, out=out)
    for i in range(9):
        for t, s in ((q, 10), (k, 20), (v, 30)):
            t.copy_(rand(t.shape, "f16", s + i))
        if i == 3:
            kv.trim(ints(2))          # idle, then growing anew
        if i == 5:
            kv.trim(ints(1, 3), ints(100, 400))  # shorter: fewer pages shared
        if i == 7:
            kv.trim(ints(2))
            kv.fork([0], [2])
        graph.replay()
        want = kv.attend_shared(q)
        torch.cuda.synchronize()
        assert torch.equal(out, want), i
        ref = KO.Cache(np64(kv.pool), kv.tables.cpu().numpy(), kv.lens.cpu().numpy(), kv.refs.cpu().numpy())
        full = ref.attend(0, [0, 1, 2, 3], [1] * 4, np64(q), 0.125)
        assert np.abs(np64(out) - full).max() <= 2e-3 * np.abs(full).max()
    kv.check()
