"""Norm, rotary append, shared attention and sampling together, as a decode step uses them: the example's model on a
cache whose every call is compared with the oracles', and steps that end in sampled tokens."""
from __future__ import annotations

import importlib.util
import os

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from _kv import UNIT, np64  # noqa: E402
from oracle import kv_oracle as KO  # noqa: E402
from oracle import step_oracle as SO  # noqa: E402
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
    """Every rotated append and every attention against the oracles, on the cache's own state."""
    calls = [0, 0]

    def positions(self, seqs, rows):
        lens, n = self.lens.tolist(), rows // len(seqs)
        return [lens[s] - n + i for s in seqs.tolist() for i in range(n)]

    def append_rotated(self, q, k, v, rotary, *, layer=0, seqs=None, out=None, **kw):
        q0, k0, pool = q.clone(), k.clone(), self.pool.clone()
        out = super().append_rotated(q, k, v, rotary, layer=layer, seqs=seqs, out=out, **kw)
        pos, u = self.positions(seqs, len(q0)), UNIT["f16"]
        for x, got in ((q0, out), (k0, None)):
            ref = SO.rotate(np64(x), pos, rotary.freqs, rotary.size, rotary.interleaved)
            if got is None:
                where = [(int(self.tables[s, p // self.page_size]), p % self.page_size)
                         for s, p in zip(np.repeat(seqs.tolist(), len(q0) // len(seqs)), pos)]
                got = torch.stack([self.pool[a, layer, 0, :, b] for a, b in where])
                assert torch.equal(torch.stack([self.pool[a, layer, 1, :, b] for a, b in where]), v)
                for a, b in where:  # nothing else was written
                    pool[a, layer, :, :, b] = self.pool[a, layer, :, :, b]
            big = np.abs(np64(x)).max() * 2
            assert (np.abs(np64(got) - ref) <= u * np.abs(ref) + 2.0 ** -21 * big + 2.0 ** -25).all()
        assert torch.equal(pool.view(torch.int16), self.pool.view(torch.int16))
        Checked.calls[0] += 1
        return out

    def _checked(self, q, out, layer, seqs, window, sinks):
        ref = KO.Cache(self.pool.to(torch.float64).cpu().numpy(), self.tables.cpu().numpy(), self.lens.cpu().numpy(),
                       self.refs.cpu().numpy())
        slots, n = seqs.tolist(), q.shape[0] // len(seqs)
        want = ref.attend(layer, slots, [n] * len(slots), np64(q), self.head_dim ** -0.5, window, sinks)
        u, at = UNIT["f16"], 0
        for s in slots:  # as in _kv.check_out
            k, v = ref.tokens(s, layer, 0), ref.tokens(s, layer, 1)
            es = (self.head_dim + 2) * 2.0 ** -24 * np.abs(np64(q[at:at + n])).sum(2, keepdims=True) * np.abs(k).max() * self.head_dim ** -0.5
            tol = np.abs(v).max() * (u + 2 * es + (len(k) + 64) * 2.0 ** -23) + u * np.abs(want[at:at + n]) + 2.0 ** -24
            assert (np.abs(np64(out[at:at + n]) - want[at:at + n]) <= tol).all()
            at += n
        Checked.calls[1] += 1
        return out

    def attend(self, q, *, layer=0, seqs=None, window=0, sinks=0, out=None):
        out = super().attend(q, layer=layer, seqs=seqs, window=window, sinks=sinks, out=out)
        return self._checked(q, out, layer, seqs, window, sinks)

    def attend_shared(self, q, *, layer=0, seqs=None, window=0, sinks=0, out=None):
        out = super().attend_shared(q, layer=layer, seqs=seqs, window=window, sinks=sinks, out=out, least=0)
        return self._checked(q, out, layer, seqs, window, sinks)


def test_a_course_of_forked_sampled_answers(ex):
    Checked.calls[:] = [0, 0]
    model = ex.Model()
    kv = Checked(80, 16, ex.KV_HEADS, ex.HEAD_DIM, layers=2, max_seqs=4, max_pages=24)
    kv.pool.zero_()
    first = ex.prompt(model, kv, 0, torch.arange(270, device="cuda") * 37 % ex.VOCAB)
    kv.fork(ex.ints(0, 0, 0), ex.ints(1, 2, 3))  # 256 shared tokens
    tokens, seqs = (first + torch.arange(4, device="cuda")) % ex.VOCAB, ex.ints(0, 1, 2, 3)
    settings = dict(temperature=0.8, top_k=50, top_p=0.95, min_p=0.01)
    g = torch.Generator().manual_seed(1)
    for _ in range(3):
        kv.extend(ex.ints(1, 1, 1, 1))
        x = model.rows(tokens, kv, shared=True, seqs=seqs)
        logits, u = model.logits(x), torch.rand(4, generator=g).cuda()
        tokens = model.pick(x, u, **settings)
        f = {k: float(np.float32(v)) if k != "top_k" else v for k, v in settings.items()}
        want = [SO.sample(np64(logits[i]), float(u[i]), **f)[0] for i in range(4)]
        assert tokens.tolist() == want
    kv.check()
    assert Checked.calls == [2 * (9 + 3), 2 * (9 + 3)]


def test_norms_of_the_model(ex):
    """The sum that a layer leaves in the residual, and the norm of it, at the model's width."""
    g = torch.Generator().manual_seed(2)
    x, y = (torch.randn((5, ex.HIDDEN), generator=g).half().cuda() for _ in range(2))
    stream = x.clone()
    out = Q.rms_norm(y, residual=stream)
    assert torch.equal(stream, x + y)
    ref = SO.rms_norm(np64(x + y))
    assert (np.abs(np64(out) - ref) <= np.abs(ref) * (UNIT["f16"] + 2.0 ** -18) + 2.0 ** -25).all()


def test_sampled_graph_steps_equal_eager_steps(ex):
    """Replays with new uniform numbers give what eager steps with the same ones give."""
    model, pairs = ex.Model(), []
    for _ in range(2):
        kv = model.cache()
        kv.pool.zero_()
        first = ex.prompt(model, kv, 0, torch.arange(45, device="cuda") * 13 % ex.VOCAB)
        kv.fork(ex.ints(0, 0), ex.ints(1, 3))
        pairs.append(ex.Decoder(model, kv, [0, 1, 3], (first + torch.arange(3, device="cuda")) % ex.VOCAB,
                                temperature=1.5, top_k=200, top_p=0.9))
    a, b = pairs
    for i in range(8):
        torch.manual_seed(i)
        a.step()
        torch.manual_seed(i)
        b.u.uniform_()
        b.eager()
        torch.cuda.synchronize()
        assert torch.equal(a.u, b.u) and torch.equal(a.tokens, b.tokens)
        assert torch.equal(a.kv.lens, b.kv.lens) and torch.equal(a.kv.pool.view(torch.int16), b.kv.pool.view(torch.int16))
