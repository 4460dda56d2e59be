"""The many-row attention over its own edges: page sizes, tiles that blocks share
out, joins of uneven parts, layers, repeats on another stream; and the page
operations on another stream than the caller's."""
from __future__ import annotations

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from _kv import Pair, check_out, np64, rand  # noqa: E402
from test_gpu_kv_attend import run  # noqa: E402
import bit_weight_only_packed_amd as Q  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _gpu_present():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


@pytest.mark.parametrize("dtype,page", [("f16", 16), ("bf16", 32), ("f16", 64), ("bf16", 128), ("f16", 256)])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_page_sizes(D, dtype, page):
    """Pages smaller than, as large as and larger than a tile; prompts that end inside both."""
    run(Pair([97, 301], dtype, page, 1, D), [97, 140], 2)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("rows,G", [(33, 5), (129, 1), (13, 10)])
def test_joins(D, rows, G):
    """One long slot among short ones: its blocks are shared by many workgroups, the last block holds few rows, the
    others' are not shared; a slot without tokens, one without rows."""
    run(Pair([2600, rows, 0, 40, 700], "f16", 32, 1, D), [rows, rows, 7, 0, rows], G)


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("window,sinks", [(600, 5), (2000, 0), (1, 700), (130, 64)])
def test_joins_through_windows(D, window, sinks):
    """Shared blocks whose tiles are those of the sinks and of the window, apart or meeting."""
    run(Pair([2100, 150], "bf16", 16, 1, D), [90, 150], 1, window=window, sinks=sinks)


def test_many_parts():
    """One block of a long slot: over a hundred parts, more of them than a wave has lanes."""
    run(Pair([70001], "f16", 256, 1, 64), [35], 2)


@pytest.mark.parametrize("heads", [1, 3, 8])
def test_block_order_covers_every_head_and_entry(heads):
    run(Pair([65, 1, 130, 258], "f16", 16, heads, 64), [65, 1, 130, 129], 1)


def test_layers_and_columns():
    p = Pair([200, 130], "bf16", 16, 2, 128, layers=3)
    q = rand((260, 4, 128), "bf16", 3)
    wide = torch.zeros((260, 8, 128), dtype=torch.bfloat16, device="cuda")
    wide[:, 1:5] = q
    out = p.gpu.attend(wide[:, 1:5], layer=2, seqs=[0, 1])
    check_out(out, p.ref.attend(2, [0, 1], [130, 130], np64(q), 128 ** -0.5), "bf16", q, p, 2, [0, 1], [130, 130], 128 ** -0.5)


def test_shared_blocks_repeat_on_another_stream():
    p = Pair([3000, 500], "f16", 16, 2, 128)
    q = rand((200, 4, 128), "f16", 4)
    first = p.gpu.attend(q, seqs=[0, 1])
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    again = p.gpu.attend(q, seqs=[0, 1], stream=s)
    s.synchronize()
    assert torch.equal(first.view(torch.int16), again.view(torch.int16))


def test_graph_of_shared_blocks():
    """A captured many-row call and its join follow the lengths at each replay."""
    p = Pair([2000], "f16", 16, 1, 64, max_pages=160)
    q = rand((150, 2, 64), "f16", 4)
    out = p.gpu.attend(q, seqs=torch.zeros(1, dtype=torch.int32, device="cuda"))
    seqs = torch.zeros(1, dtype=torch.int32, device="cuda")
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        p.gpu.attend(q, seqs=seqs, out=out)
    for n in (2000, 1500, 150, 40, 1999):
        p.gpu.lens.fill_(n)
        p.ref.lens[0] = n
        g.replay()
        torch.cuda.synchronize()
        check_out(out, p.ref.attend(0, [0], [150], np64(q), 0.125), "f16", q, p, 0, [0], [150], 0.125)


def test_pages_and_append_on_another_stream():
    p = Pair([20, 33, 0], "f16", 16, 2, 64, extra=8, max_pages=6)
    k, v = rand((6, 2, 64), "f16", 5), rand((6, 2, 64), "f16", 6)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    p.gpu.fork([0], [2], stream=s)
    p.gpu.extend([2, 2, 2], stream=s)
    p.gpu.append(k, v, seqs=[0, 1, 2], stream=s)
    p.gpu.trim([1], [7], stream=s)
    p.gpu.compact(stream=s)
    s.synchronize()
    p.ref.fork([0], [2])
    p.ref.extend([2, 2, 2])
    p.ref.append(0, [0, 1, 2], [2, 2, 2], np64(k), np64(v))
    p.ref.trim([1], [7])
    p.ref.compact()
    p.same_state()


def test_refusals_of_outputs_and_scales():
    p = Pair([40, 9], "f16", 16, 2, 64)
    q = rand((2, 4, 64), "f16", 4)
    with pytest.raises(Q.QGError, match="too large"):
        p.gpu.attend(q, seqs=[0, 1], scale=3e38)
    for out in (torch.zeros((1, 4, 64), dtype=torch.float16, device="cuda").expand(2, 4, 64),
                torch.zeros((2, 1, 64), dtype=torch.float16, device="cuda").expand(2, 4, 64)):
        with pytest.raises(Q.QGError, match="overlap"):
            p.gpu.attend(q, seqs=[0, 1], out=out)
    # inputs may be broadcast: every head the same q
    one = rand((2, 1, 64), "f16", 7).expand(2, 4, 64)
    out = p.gpu.attend(one, seqs=[0, 1])
    assert torch.equal(out, p.gpu.attend(one.contiguous(), seqs=[0, 1]))
