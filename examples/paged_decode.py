"""Serving with packed weights and a paged key-value cache, end to end on one GPU:

    python examples/paged_decode.py

A small random-weight model (grouped-query attention, sliding window with sinks
on every second layer) takes a prompt in chunks, forks it into several answers,
decodes one token of each per step from a captured HIP graph, verifies drafted
tokens in a batch and takes back the refused ones, ends some of the answers and
moves the pages that are left together.  All products are 3-bit packed weights
(QLinear, mlp); all keys and values live in one KVCache.
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


def norm(x):
    return (x * torch.rsqrt(x.float().square().mean(-1, keepdim=True) + 1e-6)).half()


class Layer:
    def __init__(self, index: int, gen):
        self.index = index
        self.qkv = packed((Q_HEADS + 2 * KV_HEADS) * HEAD_DIM, HIDDEN, gen)
        self.o = packed(HIDDEN, Q_HEADS * HEAD_DIM, gen)
        self.gate, self.up = packed(FFN, HIDDEN, gen), packed(FFN, HIDDEN, gen)
        self.down = packed(HIDDEN, FFN, gen)
        self.mask = dict(window=24, sinks=4) if index % 2 else {}

    def __call__(self, x, kv, rows):
        y = self.qkv(norm(x)).view(x.shape[0], -1, HEAD_DIM)  # q | k | v, read where they are
        q, k, v = y.split([Q_HEADS, KV_HEADS, KV_HEADS], dim=1)
        kv.append(k, v, layer=self.index, **rows)
        a = kv.attend(q, layer=self.index, out=torch.empty(q.shape, dtype=q.dtype, device=q.device), **self.mask, **rows)
        x = x + self.o(a.view(x.shape[0], -1))
        return x + Q.mlp(self.gate, self.up, self.down, norm(x))


class Model:
    def __init__(self, layers: int = 2, seed: int = 0):
        gen = torch.Generator().manual_seed(seed)
        self.layers = [Layer(i, gen) for i in range(layers)]
        self.embed = torch.randn((VOCAB, HIDDEN), generator=gen).half().cuda()

    def cache(self, pages: int = 48, slots: int = 4, cls=Q.KVCache) -> Q.KVCache:
        return cls(pages, 16, KV_HEADS, HEAD_DIM, layers=len(self.layers), max_seqs=slots, max_pages=16)

    def rows(self, tokens, kv, **rows):
        """Hidden states of new tokens, whose room in the cache has been made."""
        x = self.embed[tokens]
        for layer in self.layers:
            x = layer(x, kv, rows)
        return x

    def pick(self, x):
        """The next token of each row."""
        return (norm(x) @ self.embed.t()).argmax(-1)


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
    """One token of every listed slot per replay of a captured graph."""

    def __init__(self, model, kv, slots, tokens):
        self.tokens = tokens.clone()
        self.grow = torch.zeros(kv.max_seqs, dtype=torch.int32, device="cuda")
        self.seqs = ints(*slots)
        self.grow[self.seqs.long()] = 1
        self.model, self.kv = model, kv
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
        self.tokens.copy_(self.model.pick(self.model.rows(self.tokens, self.kv, seqs=self.seqs)))

    def step(self):
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
    dec = Decoder(model, kv, [0, 1, 2, 3], tokens)
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
