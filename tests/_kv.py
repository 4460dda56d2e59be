"""Helpers of the key-value cache tests: seeded caches on both sides, and the
tolerances of the attention."""
from __future__ import annotations

import numpy as np
import torch

import bit_weight_only_packed_amd as Q
from oracle import kv_oracle as KO

DT = {"f16": torch.float16, "bf16": torch.bfloat16}
# unit roundoff: half a unit in the last place of 11 and 8 significant bits
UNIT = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}


def rand(shape, dtype, seed, scale=1.0, dev="cuda"):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g, dtype=torch.float64) * scale).to(DT[dtype]).to(dev)


def np64(t):
    return t.detach().cpu().to(torch.float64).numpy()


class Pair:
    """The same cache on the GPU and in the oracle: slots of given lengths on pages in a shuffled order.
    fill: value of the memory that holds no token (None: random)."""

    def __init__(self, lens, dtype="f16", page=16, heads=2, D=64, layers=1, extra=3, spare_slots=0, max_pages=None,
                 seed=1, fill=None):
        rng = np.random.default_rng(seed)
        need = [-(-n // page) for n in lens]
        pages = sum(need) + extra
        slots = len(lens) + spare_slots
        width = (max(need) + 1) if max_pages is None else max_pages
        order = rng.permutation(pages)
        tables = np.full((slots, width), -1, dtype=np.int32)
        refs = np.zeros(pages, dtype=np.int32)
        at = 0
        for s, n in enumerate(need):
            tables[s, :n] = order[at:at + n]
            refs[order[at:at + n]] = 1
            at += n
        pool = rand((pages, layers, 2, heads, page, D), dtype, seed + 1, dev="cpu")
        if fill is not None:
            junk = torch.full_like(pool, fill)
            for s, n in enumerate(lens):
                for t in range(n):
                    p = int(tables[s, t // page])
                    junk[p, :, :, :, t % page] = pool[p, :, :, :, t % page]
            pool = junk
        lens_np = np.array(list(lens) + [0] * spare_slots, dtype=np.int32)
        self.dtype = dtype
        self.gpu = Q.KVCache.of(pool.cuda(), torch.from_numpy(tables).cuda(), torch.from_numpy(lens_np).cuda(),
                                torch.from_numpy(refs).cuda())
        # the oracle moves the very bits (int16 views) and computes on their values
        self.ref = KO.Cache(pool.to(torch.float64).numpy(), tables, lens_np, refs)

    def same_state(self):
        torch.cuda.synchronize()
        assert np.array_equal(self.gpu.tables.cpu().numpy(), self.ref.tables)
        assert np.array_equal(self.gpu.lens.cpu().numpy(), self.ref.lens)
        assert np.array_equal(self.gpu.refs.cpu().numpy(), self.ref.refs)
        assert np.array_equal(np64(self.gpu.pool), self.ref.pool, equal_nan=True)


def check_out(out, ref, dtype, q, pair, layer, slots, rows, scale):
    """Every element within the bound of the arithmetic: weights rounded once (unit u times the largest |v| of the
    slot), the output rounded once (u |ref|), fp32 scores (D products of |q| |k|, twice in the exponent) and fp32 sums;
    and the errors' root mean square within 2 u of the outputs' (independent roundings of both)."""
    u = UNIT[dtype]
    o = np64(out)
    assert np.isfinite(o).all()
    at = 0
    D = q.shape[2]
    qa = np.abs(np64(q))
    for s, r in zip(slots, rows):
        k, v = pair.ref.tokens(s, layer, 0), pair.ref.tokens(s, layer, 1)
        n = k.shape[0]
        kmax = np.nanmax(np.abs(np.where(np.isfinite(k), k, 0)), initial=0.0)
        vmax = np.nanmax(np.abs(np.where(np.isfinite(v), v, 0)), initial=0.0)
        es = (D + 2) * 2.0 ** -24 * qa[at:at + r].sum(2, keepdims=True) * kmax * scale
        tol = vmax * (u + 2 * es + (n + 64) * 2.0 ** -23) + u * np.abs(ref[at:at + r]) + 2.0 ** -24
        err = np.abs(o[at:at + r] - ref[at:at + r])
        assert (err <= tol).all(), (s, float((err / tol).max()))
        at += r
    rms = np.sqrt(np.mean(ref ** 2))
    if rms > 0:
        assert np.sqrt(np.mean((o - ref) ** 2)) <= 2 * u * rms, np.sqrt(np.mean((o - ref) ** 2)) / rms
