"""What calls on the cache refuse, leave out or leave alone."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from _kv import Pair, np64, rand  # noqa: E402
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
