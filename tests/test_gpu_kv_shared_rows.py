"""Attention of shared tokens beside rows that have no output: rows left out by max_rows and rows of idle slots leave
the other rows' bits alone, whatever they hold and whatever calls went before."""
from __future__ import annotations

from types import SimpleNamespace

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from _kv import UNIT, check_out, np64, rand  # noqa: E402
from oracle import kv_oracle as KO  # noqa: E402
from test_gpu_kv_shared import Always, Forked, ints  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _gpu_present():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("D,G", [(64, 4), (128, 5), (256, 2)])
def test_left_out_rows_leave_the_others_alone(dtype, D, G):
    """Left-out rows of large scores, which would raise the running maximum of their wave; between the calls one that
    gives the same rows of a call other positions."""
    f = Forked([1500], [[30, 40, 35]], dtype, 16, 1, D, seed=16)
    kv = f.gpu
    q = rand((21, G, D), dtype, 12, 1.5)
    live = torch.zeros(21, dtype=torch.bool, device="cuda")
    live[[0, 1, 7, 8, 14, 15]] = True
    q[~live] *= 20
    kw = dict(row_start=ints(0, 7, 14, 21), max_rows=2)
    first = kv.attend_shared(q, **kw)[live]
    kv.attend_shared(rand((22, G, D), dtype, 1), seqs=ints(0, 1), row_start=ints(0, 11, 22), max_rows=11, window=20)
    assert torch.equal(kv.attend_shared(q, **kw)[live], first)
    for value in (0.0, 60000.0, float("nan"), float("inf")):
        other = q.clone()
        other[~live] = value
        assert torch.equal(kv.attend_shared(other, **kw)[live], first), value


def test_idle_rows_leave_the_others_alone():
    f = Forked([1500], [[30, 40, 35, 9]], "f16", 16, 1, 64, seed=17)
    kv = f.gpu
    kv.trim(ints(1, 2))
    q = rand((4, 8, 64), "f16", 3, 1.5)
    first = kv.attend_shared(q)
    assert (first[[1, 2]] == 0).all()
    for value in (0.0, 60000.0, float("nan")):
        other = q.clone()
        other[[1, 2]] = value
        got = kv.attend_shared(other)
        assert torch.equal(got[[0, 3]], first[[0, 3]]) and (got[[1, 2]] == 0).all(), value


def test_groups_that_hold_nothing_are_refused():
    """Not taken for no groups at all, which is one of all entries."""
    f = Forked([640], [[2, 9, 5]], "f16", 16, 1, 64, seed=18)
    q = rand((3, 4, 64), "f16", 4)
    for groups in ([], torch.empty(0, dtype=torch.int32, device="cuda")):
        with pytest.raises(ValueError, match="groups"):
            f.gpu.attend_shared(q, groups=groups)
    assert f.gpu.attend_shared(q, groups=[0, 3]).shape == q.shape


@pytest.mark.parametrize("rows", [1, 3])
def test_more_entries_than_the_plan_has_threads(rows):
    """700 entries in two groups and some idle ones: a thread of the plan has several."""
    n = 700
    kv = Always(40 + 2 * n, 16, 1, 64, max_seqs=n + 1, max_pages=24)
    kv.extend([0] * n + [320])
    kv.append(rand((320, 1, 64), "f16", 1), rand((320, 1, 64), "f16", 2), seqs=[n])
    kv.fork([n] * n, list(range(n)))
    grow = torch.randint(rows, 9, (n + 1,), generator=torch.Generator().manual_seed(3), dtype=torch.int32)
    grow[n] = 0
    kv.extend(grow.cuda())
    total = int(grow.sum())
    start = torch.zeros(n + 1, dtype=torch.int32)
    start[1:] = grow[:n].cumsum(0)
    kv.append(rand((total, 1, 64), "f16", 4), rand((total, 1, 64), "f16", 5), seqs=list(range(n)), row_start=start.cuda(), max_rows=8)
    kv.trim([5, 300, 699])
    kv.check()
    q = rand((n * rows, 2, 64), "f16", 6, 1.5)
    seqs = torch.arange(n, dtype=torch.int32, device="cuda")
    got = kv.attend_shared(q, seqs=seqs, groups=[0, 333, n])
    plain = kv.attend(q, seqs=seqs)
    assert not torch.equal(got, plain)
    # both within 2 u of the definition in the root mean square, and some of them against it
    err = (got.double() - plain.double()).square().mean().sqrt()
    assert err <= 4 * UNIT["f16"] * plain.double().square().mean().sqrt()
    ref = KO.Cache(np64(kv.pool), kv.tables.cpu().numpy(), kv.lens.cpu().numpy(), kv.refs.cpu().numpy())
    for s in (0, 5, 255, 256, 332, 333, 511, 512, 699):
        mine = slice(s * rows, (s + 1) * rows)
        check_out(got[mine], ref.attend(0, [s], [rows], np64(q[mine]), 0.125), "f16", q[mine], SimpleNamespace(ref=ref), 0, [s], [rows], 0.125)
