"""Serving with packed weights and a paged key-value cache, end to end on one GPU:

    python examples/paged_decode.py

A small random-weight model (grouped-query attention with rotary positions, sliding
window with sinks on every second layer) takes a prompt in chunks, forks it into
several answers, decodes one sampled token of each per step from a captured HIP
graph, verifies drafted tokens in a batch and takes back the refused ones, ends some
of the answers and moves the pages that are left together.  All products are 3-bit
packed weights (QLinear, mlp); all keys and values live in one KVCache; norms,
rotation and sampling are the library's (rms_norm, Rotary, sample).
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import bit_weight_only_packed_amd as Q  # noqa: E402

HIDDEN, Q_HEADS, KV_HEADS, HEAD_DIM, FFN, VOCAB = 1280, 10, 2, 128, 2560, 1024
MAX_ROWS = 32  # rows of a call of the packed products


def packed(n: int, k: int, gen) -> Q.QLinear:
    """A random 3-bit matrix whose products keep the size of their inputs."""
    codes = torch.randint(-2 ** 31, 2 ** 31 - 1, (n * k * 3 // 32,), dtype=torch.int32, generator=gen).cuda()
    scales = torch.full((n, k // Q.GROUP), 1 / (2.29 * k ** 0.5), dtype=torch.float16).cuda()  # codes' deviation 2.29
    return Q.QLinear(codes, scales, k, n, bits=3, max_M=MAX_ROWS)


class Layer:
    def __init__(self, index: int, gen, rotary):
        self.index, self.rotary = index, rotary
        self.qkv = packed((Q_HEADS + 2 * KV_HEADS) * HEAD_DIM, HIDDEN, gen)
        self.o = packed(HIDDEN, Q_HEADS * HEAD_DIM, gen)
        self.gate, self.up = packed(FFN, HIDDEN, gen), packed(FFN, HIDDEN, gen)
        self.down = packed(HIDDEN, FFN, gen)
        self.mask = dict(window=24, sinks=4) if index % 2 else {}

    def __call__(self, x, kv, rows, shared=False):
        y = self.qkv(Q.rms_norm(x)).view(x.shape[0], -1, HEAD_DIM)  # q | k | v, read where they are
        q, k, v = y.split([Q_HEADS, KV_HEADS, KV_HEADS], dim=1)
        kv.append_rotated(q, k, v, self.rotary, layer=self.index, out=q, **rows)
        attend = kv.attend_shared if shared else kv.attend
        a = attend(q, layer=self.index, out=torch.empty(q.shape, dtype=q.dtype, device=q.device), **self.mask, **rows)
        y = Q.rms_norm(self.o(a.view(x.shape[0], -1)), residual=x)  # x holds the sum
        return x + Q.mlp(self.gate, self.up, self.down, y)


class Model:
    def __init__(self, layers: int = 2, seed: int = 0):
        gen = torch.Generator().manual_seed(seed)
        rotary = Q.Rotary(HEAD_DIM)
        self.layers = [Layer(i, gen, rotary) for i in range(layers)]
        self.embed = torch.randn((VOCAB, HIDDEN), generator=gen).half().cuda()

    def cache(self, pages: int = 48, slots: int = 4, cls=Q.KVCache) -> Q.KVCache:
        return cls(pages, 16, KV_HEADS, HEAD_DIM, layers=len(self.layers), max_seqs=slots, max_pages=16)

    def rows(self, tokens, kv, shared=False, **rows):
        """Hidden states of new tokens, whose room in the cache has been made.  shared: the rows' slots may hold
        the same pages, as forked answers do."""
        x = self.embed[tokens]
        for layer in self.layers:
            x = layer(x, kv, rows, shared)
        return x

    def logits(self, x):
        return Q.rms_norm(x) @ self.embed.t()

    def pick(self, x, u=None, **settings):
        """The next token of each row: the likeliest, or by uniform numbers u and the settings of sample."""
        if u is None:
            u, settings = torch.zeros(x.shape[0], device=x.device), dict(temperature=0.0)
        return Q.sample(self.logits(x), u, **settings).long()


def ints(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def prompt(model, kv, slot: int, tokens):
    """A prompt, in chunks of the rows that the packed products take; returns the token that follows it."""
    grow, seqs = torch.zeros(kv.max_seqs, dtype=torch.int32, device="cuda"), ints(slot)
    for part in tokens.split(MAX_ROWS):
        grow[slot] = len(part)
        kv.extend(grow)
        x = model.rows(part, kv, seqs=seqs)
    return model.pick(x[-1:])


class Decoder:
    """One token of every listed slot per replay of a captured graph: the likeliest, or with settings of ``sample`` by
    uniform numbers drawn before each."""

    def __init__(self, model, kv, slots, tokens, **settings):
        self.tokens = tokens.clone()
        self.grow = torch.zeros(kv.max_seqs, dtype=torch.int32, device="cuda")
        self.seqs = ints(*slots)
        self.grow[self.seqs.long()] = 1
        self.model, self.kv, self.settings = model, kv, settings
        self.u = torch.zeros(len(slots), device="cuda") if settings else None
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):  # what is made once (workspaces of the library calls) is made before the capture
            model.pick(model.embed[self.tokens])
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph):
            self.eager()

    def eager(self):
        self.kv.extend(self.grow)
        x = self.model.rows(self.tokens, self.kv, shared=True, seqs=self.seqs)
        self.tokens.copy_(self.model.pick(x, self.u, **self.settings))

    def step(self):
        if self.u is not None:
            self.u.uniform_()
        self.graph.replay()
        return self.tokens


def verify(model, kv, slots, tokens, drafts):
    """Each slot's last token and its drafts [slots][n] in one batch: the drafts up to the first that the model
    would not have picked are kept, the others' keys and values taken back.  Returns the kept counts and the
    token that follows each."""
    n = drafts.shape[1]
    grow = torch.zeros(kv.max_seqs, dtype=torch.int32, device="cuda")
    seqs = ints(*slots)
    grow[seqs.long()] = n + 1
    had = kv.lens[seqs.long()].clone()
    kv.extend(grow)
    rows = torch.cat([tokens[:, None], drafts], 1)
    picked = model.pick(model.rows(rows.reshape(-1), kv, seqs=seqs)).view(-1, n + 1)
    kept = (picked[:, :n] == drafts).int().cumprod(1).sum(1).int()
    kv.trim(seqs, had + 1 + kept)
    return kept, picked.gather(1, kept.long()[:, None])[:, 0]


def main():
    model = Model()
    kv = model.cache()
    first = prompt(model, kv, 0, torch.arange(70, device="cuda") * 37 % VOCAB)
    kv.fork(ints(0, 0, 0), ints(1, 2, 3))  # four answers to one prompt
    tokens = (first + torch.arange(4, device="cuda")) % VOCAB
    torch.manual_seed(0)
    dec = Decoder(model, kv, [0, 1, 2, 3], tokens, temperature=0.8, top_k=50, top_p=0.95)
    for _ in range(20):
        tokens = dec.step()
    kept, tokens = verify(model, kv, [0, 1, 2, 3], tokens, torch.randint(0, VOCAB, (4, 7), device="cuda"))
    kv.trim(ints(0, 2))  # two answers end
    kv.compact()
    dec = Decoder(model, kv, [1, 3], tokens[[1, 3]])
    for _ in range(10):
        tokens = dec.step()
    kv.check()
    print("lengths", kv.lens.tolist(), "kept drafts", kept.tolist(), "live pages", int((kv.refs > 0).sum()),
          "tokens", tokens.tolist())


if __name__ == "__main__":
    main()
