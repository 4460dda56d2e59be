"""The example that runs the packed products and the cache together: every
attention of it against the oracle, its graph replays against eager steps bit for
bit, its pages' bookkeeping, and its whole course."""
from __future__ import annotations

import importlib.util
import os

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from _kv import UNIT, np64  # noqa: E402
from oracle import kv_oracle as KO  # noqa: E402
import bit_weight_only_packed_amd as Q  # noqa: E402

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "paged_decode.py")


@pytest.fixture(scope="module")
def ex():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    spec = importlib.util.spec_from_file_location("paged_decode", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


class Checked(Q.KVCache):
    """A cache whose every attend is compared with the oracle's on the cache's own state."""
    calls = 0

    def attend(self, q, *, layer=0, seqs=None, window=0, sinks=0, out=None, **kw):
        out = super().attend(q, layer=layer, seqs=seqs, window=window, sinks=sinks, out=out, **kw)
        ref = KO.Cache(self.pool.to(torch.float64).cpu().numpy(), self.tables.cpu().numpy(), self.lens.cpu().numpy(),
                       self.refs.cpu().numpy())
        slots, n = seqs.tolist(), q.shape[0] // len(seqs)
        want = ref.attend(layer, slots, [n] * len(slots), np64(q), self.head_dim ** -0.5, window, sinks)
        err = np.abs(np64(out) - want)
        # one rounding of the weights, one of the output, fp32 scores (see _kv.check_out)
        u, at = UNIT["f16"], 0
        for s in slots:
            k, v = ref.tokens(s, layer, 0), ref.tokens(s, layer, 1)
            es = (self.head_dim + 2) * 2.0 ** -24 * np.abs(np64(q[at:at + n])).sum(2, keepdims=True) \
                * np.abs(k).max() * self.head_dim ** -0.5
            tol = np.abs(v).max() * (u + 2 * es + (len(k) + 64) * 2.0 ** -23) + u * np.abs(want[at:at + n]) + 2.0 ** -24
            assert (err[at:at + n] <= tol).all()
            at += n
        Checked.calls += 1
        return out


def test_every_attention_of_the_course(ex):
    Checked.calls = 0
    model = ex.Model()
    kv = model.cache(cls=Checked)
    first = ex.prompt(model, kv, 0, torch.arange(70, device="cuda") * 37 % ex.VOCAB)
    kv.fork(ex.ints(0, 0), ex.ints(1, 2))
    tokens = (first + torch.arange(3, device="cuda")) % ex.VOCAB
    drafts = torch.arange(21, device="cuda").view(3, 7) * 11 % ex.VOCAB
    kept, tokens = ex.verify(model, kv, [0, 1, 2], tokens, drafts)
    assert torch.equal(kv.lens[:3], 71 + kept)
    kv.trim(ex.ints(1))
    kv.compact()
    grow = ex.ints(1, 0, 1, 0)
    for _ in range(3):
        kv.extend(grow)
        tokens = model.pick(model.rows(tokens[[0, 2]] if len(tokens) == 3 else tokens, kv, seqs=ex.ints(0, 2)))
    kv.check()
    assert Checked.calls == 2 * (3 + 1 + 3)
    live = int((kv.refs > 0).sum())
    assert (kv.refs[:live] > 0).all() and int(kv.info[2]) <= live
    named = kv.tables[kv.tables >= 0].long()
    assert torch.equal(torch.bincount(named, minlength=kv.pages).int(), kv.refs)


def test_graph_steps_equal_eager_steps(ex):
    """Replays give the tokens, lengths, tables and pool that eager steps give on a cache of the same state."""
    model = ex.Model()
    kvs, tokens = [], None
    for _ in range(2):
        kv = model.cache()
        kv.pool.zero_()
        first = ex.prompt(model, kv, 0, torch.arange(45, device="cuda") * 13 % ex.VOCAB)
        kv.fork(ex.ints(0, 0), ex.ints(1, 3))
        tokens = (first + torch.arange(3, device="cuda")) % ex.VOCAB
        kvs.append(kv)
    a = ex.Decoder(model, kvs[0], [0, 1, 3], tokens)
    b = ex.Decoder(model, kvs[1], [0, 1, 3], tokens)
    for _ in range(8):
        a.step()
        b.eager()
        torch.cuda.synchronize()
        assert torch.equal(a.tokens, b.tokens)
        assert torch.equal(kvs[0].lens, kvs[1].lens) and torch.equal(kvs[0].tables, kvs[1].tables)
        assert torch.equal(kvs[0].pool.view(torch.int16), kvs[1].pool.view(torch.int16))


def test_the_example_runs(ex, capsys):
    ex.main()
    assert "lengths [0, " in capsys.readouterr().out
