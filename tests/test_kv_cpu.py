"""The paged key-value cache without a GPU: refusals of the C ABI, the binding's
constants against include/qgkv.h, and the oracle's own pins (closed forms, brute
force and invariants of the page operations)."""
from __future__ import annotations

import contextlib
import ctypes
import re
import types

import numpy as np
import pytest

import bit_weight_only_packed_amd as Q
from bit_weight_only_packed_amd import kv_cache as B
from oracle import kv_oracle as KO


@pytest.fixture(scope="module")
def L():
    return Q.lib()


def _desc(**kw):
    d = B._KvDesc(64, 2, 8, 128, 16, 4, 32, B.TYPE_F16, 0x100000, 0x200000, 0x300000, 0x400000, 0x500000)
    for k, v in kw.items():
        setattr(d, k, v)  # never dereferenced: validation fails first
    return d


@pytest.mark.parametrize("kw,status,frag", [
    (dict(pages=0), 1, "pages"), (dict(pages=(1 << 20) + 1), 1, "pages"), (dict(layers=0), 1, "layers"),
    (dict(kv_heads=0), 1, "kv_heads"), (dict(kv_heads=1025), 1, "kv_heads"),
    (dict(head_dim=96), 2, "head_dim"), (dict(head_dim=0), 2, "head_dim"),
    (dict(page_size=8), 1, "page_size"), (dict(page_size=48), 1, "page_size"), (dict(page_size=512), 1, "page_size"),
    (dict(page_size=0), 1, "page_size"), (dict(page_size=-16), 1, "page_size"),
    (dict(max_seqs=0), 1, "max_seqs"), (dict(max_seqs=1025), 1, "max_seqs"),
    (dict(max_pages=0), 1, "max_pages"), (dict(max_pages=(1 << 26) + 1), 1, "max_pages"), (dict(dtype=2), 1, "dtype"),
    (dict(pool=None), 1, "pool"), (dict(tables=None), 1, "tables"), (dict(info=None), 1, "info"),
    (dict(pool=0x100008), 1, "aligned"), (dict(refs=0x400004), 1, "aligned"), (dict(lens=0x300002), 1, "aligned"),
])
def test_create_refuses(L, kw, status, frag):
    want = {1: Q.QG_ERR_INVALID_ARG, 2: Q.QG_ERR_UNSUPPORTED}[status]
    h = ctypes.c_void_p(1)
    d = _desc(**kw)
    assert L.qgkv_create(ctypes.byref(h), ctypes.byref(d), None) == want
    assert h.value is None
    assert frag in L.qg_last_error().decode()


def test_null_arguments(L):
    d, h = _desc(), ctypes.c_void_p()
    b, r = B._KvBatch(1, 1, 1, None, None), B._KvRows(0x1000, 128, 128)
    assert L.qgkv_create(None, ctypes.byref(d), None) == Q.QG_ERR_INVALID_ARG
    assert L.qgkv_create(ctypes.byref(h), None, None) == Q.QG_ERR_INVALID_ARG
    b, r = ctypes.byref(b), ctypes.byref(r)
    for st in (L.qgkv_extend(None, 0x1000, None), L.qgkv_fork(None, 0x1000, 0x1000, 1, None),
               L.qgkv_trim(None, 0x1000, None, 1, None), L.qgkv_compact(None, None),
               L.qgkv_append(None, 0, b, r, r, None), L.qgkv_attend(None, 0, b, r, r, 8, 1.0, 0, 0, None)):
        assert st == Q.QG_ERR_INVALID_ARG
        assert "handle" in L.qg_last_error().decode()
    assert L.qgkv_destroy(None) == Q.QG_OK


def test_binding_constants_match_the_header():
    text = open(Q.KV_HEADER_PATH).read()
    decl = {n: int(v) for n, v in re.findall(r"\b(QG_KV_[A-Z0-9_]+)\s*=\s*(\d+)", text)}
    assert decl == {"QG_KV_F16": B.TYPE_F16, "QG_KV_BF16": B.TYPE_BF16, "QG_KV_SHORT": B.INFO_SHORT,
                    "QG_KV_LONG": B.INFO_LONG, "QG_KV_PAIR": B.INFO_PAIR, "QG_KV_MAX_SEQS": B.MAX_SEQS,
                    "QG_KV_MIN_PAGE": B.MIN_PAGE, "QG_KV_MAX_PAGE": B.MAX_PAGE}
    assert (KO.SHORT, KO.LONG, KO.PAIR) == (B.INFO_SHORT, B.INFO_LONG, B.INFO_PAIR)


def test_descriptor_fields_match_the_header():
    text = open(Q.KV_HEADER_PATH).read()
    for struct, cls in (("qg_kv_desc", B._KvDesc), ("qg_kv_batch", B._KvBatch), ("qg_kv_rows", B._KvRows)):
        body = re.search(r"typedef struct \{([^}]*)\} %s;" % struct, text).group(1)
        body = re.sub(r"/\*.*?\*/", "", body, flags=re.S)
        assert re.findall(r"(\w+);", body) == [f[0] for f in cls._fields_]


# ---- the oracle ----------------------------------------------------------------
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (3, 0), (3, 2), (4, 9), (100, 1)])
def test_sees_counts(window, sinks):
    """How many of n tokens a row sees, in closed form."""
    for pos in range(-3, 12):
        n = sum(KO.sees(pos, t, window, sinks) for t in range(20))
        first = 0 if window == 0 else max(pos - window + 1, 0)
        assert n == (0 if pos < 0 else pos + 1 - first + min(first, sinks if window else 0))


def test_attention_of_equal_scores_is_the_mean():
    v = np.arange(12.0).reshape(6, 2)
    assert np.allclose(KO.attend_row(np.zeros(4), np.ones((6, 4)), v, 3, 1.0), v[:4].mean(0))
    assert np.allclose(KO.attend_row(np.zeros(4), np.ones((6, 4)), v, 5, 1.0, 2, 1), v[[0, 4, 5]].mean(0))
    assert (KO.attend_row(np.zeros(4), np.ones((6, 4)), v, -1, 1.0) == 0).all()


def test_attention_of_known_weights():
    """q . k = log w gives weights w / sum w; a shift of all scores changes nothing."""
    w = np.array([1.0, 2.0, 5.0])
    k, v = np.log(w)[:, None], np.eye(3)
    assert np.allclose(KO.attend_row([1.0], k, v, 2, 1.0), w / 8, rtol=1e-15)
    assert np.allclose(KO.attend_row([1.0], k + 700, v, 2, 1.0), w / 8, rtol=1e-12)
    assert np.allclose(KO.attend_row([2.0], k, v, 2, 0.5), w / 8, rtol=1e-15)


def _cache(lens, pages=12, page=4, layers=1, heads=1, D=2, width=6):
    t = np.full((len(lens), width), -1, dtype=np.int64)
    refs, at = np.zeros(pages, dtype=np.int64), 0
    for s, n in enumerate(lens):
        for i in range(-(-n // page)):
            t[s, i], refs[at] = at, 1
            at += 1
    pool = np.random.default_rng(3).standard_normal((pages, layers, 2, heads, page, D))
    return KO.Cache(pool, t, np.array(lens), refs)


def test_append_then_tokens():
    c = _cache([3, 0])
    before = c.tokens(0, 0, 0).copy()
    c.extend([3, 2])
    k, v = np.random.default_rng(1).standard_normal((2, 5, 1, 2))
    c.append(0, [1, 0], [2, 3], k, v)
    assert np.array_equal(c.tokens(0, 0, 0), np.concatenate([before, k[2:]]))
    assert np.array_equal(c.tokens(1, 0, 1), v[:2])


@pytest.mark.parametrize("seed", range(8))
def test_page_operations_keep_their_invariants(seed):
    """Random lives against a plain list of tokens per slot: contents follow, counts are the tables', no page is
    both free and named, slots never see each other's writes."""
    rng = np.random.default_rng(seed)
    c = _cache([5, 8, 0, 0, 0], pages=14)
    plain = [[tuple(x[0]) for x in c.tokens(s, 0, 0)] for s in range(5)]
    for _ in range(60):
        op = rng.integers(4)
        if op == 0:
            n = rng.integers(0, 4, 5) * (rng.random(5) < 0.5)
            c.info[0] = 0
            c.extend(n)
            if c.info[0]:
                continue
            rows = [int(x) for x in n]
            k = rng.standard_normal((sum(rows), 1, 2))
            c.append(0, range(5), rows, k, k)
            at = 0
            for s, r in enumerate(rows):
                plain[s] += [tuple(x[0]) for x in k[at:at + r]]
                at += r
        elif op == 1:
            s, d = rng.integers(0, 5, 2)
            if s != d and not plain[d]:
                plain[d] = list(plain[s])
            c.fork([s], [d])
        elif op == 2:
            s, keep = rng.integers(0, 5), int(rng.integers(0, 12))
            c.trim([s], [keep])
            plain[s] = plain[s][:keep]
        else:
            c.compact()
            live = np.flatnonzero(c.refs)
            assert np.array_equal(live, np.arange(live.size))
        for s in range(5):
            assert [tuple(x[0]) for x in c.tokens(s, 0, 0)] == plain[s]
        named = c.tables[c.tables >= 0]
        assert np.array_equal(np.bincount(named, minlength=14), c.refs)


def test_extend_counts_what_is_short():
    c = _cache([5, 8], pages=5)
    c.extend([12, 4])
    assert c.info[:2] == [KO.SHORT, 3 + 1 - 1] and list(c.lens) == [5, 8]
    c.extend([100, 0])
    assert c.info[0] == KO.SHORT | KO.LONG


def test_append_after_a_refused_extend():
    c = _cache([5, 8], pages=5)
    before = c.pool.copy()
    k = np.ones((2, 1, 2))
    c.extend([12, 4])
    c.append(0, [0, 1], [1, 1], k, k)
    assert np.array_equal(before, c.pool)
    c.extend([1, 0])
    c.append(0, [0], [1], k[:1], k[:1])
    assert list(c.lens) == [6, 8] and (c.tokens(0, 0, 0)[5] == 1).all()
    c.extend([12, 4])
    c.info[0] = 0
    c.append(0, [1], [1], k[:1], k[:1])
    assert (c.tokens(1, 0, 0)[7] == 1).all()


@pytest.mark.parametrize("current", [0, 1])
def test_calls_run_on_the_caches_gpu(current):
    """The library refuses a cache that is not on the current GPU: a call then makes the cache's the current one for its
    time."""
    class Cuda:
        at = current

        def current_device(self):
            return self.at

        @contextlib.contextmanager
        def device(self, i):
            before, self.at = self.at, i
            yield
            self.at = before

    cuda, seen = Cuda(), []
    kv = Q.KVCache.__new__(Q.KVCache)
    kv._h, kv._dev, kv._torch = None, 1, types.SimpleNamespace(cuda=cuda)
    kv._check = lambda st: seen.append(st) if st else None

    def compact(h, st):
        seen.append((cuda.at, st))
        return Q.QG_OK if cuda.at == 1 and st == 7 else Q.QG_ERR_INVALID_ARG

    kv._c = {"compact": compact}
    kv._call("compact", 7)
    assert seen == [(0, 7)] * (current == 0) + [(1, 7)] and cuda.at == current
    kv._call("compact", 8)
    assert seen[-1] == Q.QG_ERR_INVALID_ARG and cuda.at == current
