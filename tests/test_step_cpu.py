"""Norm, rotary positions and sampling without a GPU: refusals of the C ABI, the binding's
constants against include/qgstep.h, the frequencies, and the oracle's own pins."""
from __future__ import annotations

import ctypes
import math
import re

import numpy as np
import pytest

import bit_weight_only_packed_amd as Q
from bit_weight_only_packed_amd import step_ops as B
from oracle import step_oracle as SO

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def L():
    return Q.lib()


def refused(L, status, frag):
    assert status in (Q.QG_ERR_INVALID_ARG, Q.QG_ERR_UNSUPPORTED)
    assert frag in L.qg_last_error().decode()


def norm(**kw):
    d = B._Norm(0x100000, 0x200000, 0x300000, 0x400000, None, 64, 64, 64, 4, 64, B.TYPE_F16, B.CODES_SAME, 0, 1e-6)
    for k, v in kw.items():
        setattr(d, k, v)  # never dereferenced: validation fails first
    return d


@pytest.mark.parametrize("kw,frag", [
    (dict(rows=-1), "rows"), (dict(n=0), "n ="), (dict(n=32769), "n ="), (dict(dtype=2), "dtype"), (dict(dtype=-1), "dtype"),
    (dict(codes=3), "codes"), (dict(codes=-1), "codes"), (dict(eps=0.0), "eps"), (dict(eps=-1.0), "eps"),
    (dict(eps=float("nan")), "eps"), (dict(eps=float("inf")), "eps"), (dict(group=32), "group"),
    (dict(codes=1, scales=0x500000, group=16), "group"), (dict(codes=1, scales=0x500000, group=-32), "group"),
    (dict(x=None), "x and out"), (dict(out=None), "x and out"), (dict(x=0x100001), "aligned"), (dict(weight=0x300001), "aligned"),
    (dict(codes=1), "scales"), (dict(codes=2, scales=0x500002), "scales"), (dict(x_stride=-64), "x_stride"),
    (dict(out_stride=63), "out_stride"), (dict(residual_stride=0), "residual_stride"), (dict(out=0x100002), "out overlaps x"),
    (dict(out=0x100000, out_stride=128), "out overlaps x"), (dict(residual=0x100000), "residual overlaps"),
    (dict(residual=0x400080), "residual overlaps"), (dict(weight=0x400000), "weight overlaps"),
    (dict(weight=0x200010), "weight overlaps"), (dict(codes=1, scales=0x300000), "scales overlap"),
    (dict(codes=1, out=0x100000, scales=0x500000), "out overlaps x"),
])
def test_norm_refuses(L, kw, frag):
    refused(L, L.qgs_rms_norm(ctypes.byref(norm(**kw)), None), frag)


def test_norm_of_no_rows(L):
    assert L.qgs_rms_norm(ctypes.byref(norm(rows=0, x=None, out=None)), None) == Q.QG_OK
    assert L.qgs_rms_norm(None, None) == Q.QG_ERR_INVALID_ARG


@pytest.mark.parametrize("kw,rot,frag", [
    (dict(rows=-1), {}, "rows"), (dict(heads=0), {}, "heads"), (dict(head_dim=120), {}, "head_dim"),
    (dict(head_dim=1040), {}, "head_dim"), (dict(head_dim=0), {}, "head_dim"), (dict(dtype=2), {}, "dtype"),
    ({}, dict(turns=None), "turns"), ({}, dict(turns=0x100008), "turns"), ({}, dict(dim=0), "dim"), ({}, dict(dim=24), "dim"),
    ({}, dict(dim=144), "dim"), ({}, dict(layout=2), "layout"), ({}, dict(size=float("inf")), "size"),
    (dict(x=None), {}, "x and out"), (dict(out=0x400008), {}, "x and out"), (dict(positions=None), {}, "positions"),
    (dict(x_row=1028), {}, "strides"), (dict(out_head=-128), {}, "strides"), (dict(out=0x200010), {}, "out overlaps x"),
    (dict(out_row=120), {}, "overlap"), (dict(out=0x200000, out_row=2048), {}, "out overlaps x"),
    (dict(out=0x200000, x_row=128, out_row=128, x_head=128, out_head=128), {}, "overlap"),
])
def test_rotate_refuses(L, kw, rot, frag):
    d = B._Rows(0x200000, 0x400000, 0x600000, 1024, 128, 1024, 128, 5, 8, 128, B.TYPE_F16)
    r = B._Rotary(0x100000, 128, B.HALVES, 1.0)
    for k, v in kw.items():
        setattr(d, k, v)
    for k, v in rot.items():
        setattr(r, k, v)
    refused(L, L.qgs_rotate(ctypes.byref(d), ctypes.byref(r), None), frag)


def test_rotate_nulls(L):
    d = B._Rows(None, None, None, 0, 0, 0, 0, 0, 8, 128, B.TYPE_F16)
    r = B._Rotary(0x100000, 128, B.HALVES, 1.0)
    assert L.qgs_rotate(ctypes.byref(d), ctypes.byref(r), None) == Q.QG_OK  # no rows
    assert L.qgs_rotate(None, ctypes.byref(r), None) == Q.QG_ERR_INVALID_ARG
    assert L.qgs_rotate(ctypes.byref(d), None, None) == Q.QG_ERR_INVALID_ARG


@pytest.mark.parametrize("kw,frag", [
    (dict(rows=-1), "rows"), (dict(vocab=0), "vocab"), (dict(vocab=(1 << 20) + 1), "vocab"), (dict(dtype=3), "dtype"),
    (dict(logits=None), "logits"), (dict(u=None), "logits"), (dict(tokens=None), "logits"), (dict(logits=0x100001), "aligned"),
    (dict(dtype=2, logits=0x100002), "aligned"), (dict(stride=-1), "stride"), (dict(top_k=0x200002), "aligned"),
    (dict(probs=0x200001), "aligned"),
])
def test_sample_refuses(L, kw, frag):
    d = B._Sampling(0x100000, 1000, 4, 1000, B.TYPE_F16, 0x200000, None, None, None, None, 1.0, 0, 1.0, 0.0, 0x300000, None)
    for k, v in kw.items():
        setattr(d, k, v)
    refused(L, L.qgs_sample(ctypes.byref(d), 0x400000, 1 << 24, None), frag)


def test_sample_workspace(L):
    n = ctypes.c_size_t()
    assert L.qgs_sample_workspace(3, 1000, ctypes.byref(n)) == Q.QG_OK and n.value > 0
    assert Q.sample_workspace(3, 1000) == n.value
    assert L.qgs_sample_workspace(0, 1000, ctypes.byref(n)) == Q.QG_OK and n.value == 0
    refused(L, L.qgs_sample_workspace(1, 0, ctypes.byref(n)), "vocab")
    assert L.qgs_sample_workspace(1, 1000, None) == Q.QG_ERR_INVALID_ARG
    d = B._Sampling(0x100000, 1000, 4, 1000, B.TYPE_F16, 0x200000, None, None, None, None, 1.0, 0, 1.0, 0.0, 0x300000, None)
    need = Q.sample_workspace(4, 1000)
    refused(L, L.qgs_sample(ctypes.byref(d), 0x400000, need - 1, None), "workspace")
    refused(L, L.qgs_sample(ctypes.byref(d), 0x400008, need, None), "workspace")
    refused(L, L.qgs_sample(ctypes.byref(d), None, need, None), "workspace")
    assert L.qgs_sample(None, 0x400000, need, None) == Q.QG_ERR_INVALID_ARG


def test_cache_calls_without_a_cache(L):
    from bit_weight_only_packed_amd import kv_cache as K
    b, r = ctypes.byref(K._KvBatch(1, 1, 1, None, None)), ctypes.byref(K._KvRows(0x1000, 128, 128))
    rot = ctypes.byref(B._Rotary(0x100000, 128, B.HALVES, 1.0))
    refused(L, L.qgkv_append_rotary(None, 0, b, r, r, r, r, 8, rot, None), "handle")
    refused(L, L.qgkv_attend_shared(None, 0, b, r, r, 8, 1.0, 0, 0, None, 1, -1, None), "handle")


def test_binding_refuses_before_the_library():
    x = torch.zeros((2, 16), dtype=torch.float16)
    with pytest.raises(ValueError, match="GPU"):
        Q.rms_norm(x)
    with pytest.raises(ValueError, match="GPU"):
        Q.sample(x, torch.zeros(2))
    with pytest.raises(ValueError, match="dim"):
        Q.Rotary(24, device="cpu")
    with pytest.raises(ValueError, match="scaling"):
        Q.Rotary(32, scaling="other", device="cpu")
    with pytest.raises(ValueError, match="yarn"):
        Q.Rotary(32, scaling="yarn", factor=2.0, fast=1.0, slow=2.0, device="cpu")
    with pytest.raises(ValueError, match="base"):
        Q.Rotary(32, base=1.0, device="cpu")
    with pytest.raises(ValueError, match="freqs"):
        Q.Rotary.of([1.0] * 7, device="cpu")
    with pytest.raises(ValueError, match="GPU"):
        Q.Rotary(16, device="cpu").rotate(x[:, None], torch.zeros(2, dtype=torch.int32))


def test_binding_constants_match_the_header():
    text = open(Q.STEP_HEADER_PATH).read()
    decl = {}
    for name, expr in re.findall(r"\b(QGS_[A-Z0-9_]+)\s*=\s*(\d+(?:\s*<<\s*\d+)?)", text):
        a, _, b = expr.partition("<<")
        decl[name] = int(a) << int(b or 0)
    assert decl == {"QGS_F16": B.TYPE_F16, "QGS_BF16": B.TYPE_BF16, "QGS_F32": B.TYPE_F32, "QGS_SAME": B.CODES_SAME,
                    "QGS_INT8": B.CODES_INT8, "QGS_E4M3": B.CODES_E4M3, "QGS_MAX_NORM": B.MAX_NORM,
                    "QGS_MAX_VOCAB": B.MAX_VOCAB, "QGS_HALVES": B.HALVES, "QGS_PAIRS": B.PAIRS}


# ------------------------------------------------------------------------------------------------- frequencies

def turns(r):
    return [int(w) & (2 ** 64 - 1) for w in r.turns.tolist()]


def test_turns_are_the_frequencies():
    """Each word is its frequency over 2 pi to 2^-53 of itself (a 64-bit float's rounding, twice) and 2^-64."""
    r = Q.Rotary(128, 500000.0, device="cpu")
    for w, j in zip(turns(r), range(64)):
        f = 500000.0 ** (-2 * j / 128)
        assert abs(w / 2 ** 64 - f / (2 * math.pi)) <= 3 * 2.0 ** -53 * f + 2.0 ** -64


def test_turns_past_one_and_below_zero():
    """Whole turns do not matter, and a falling angle is a rising one of the rest of the turn."""
    r = Q.Rotary.of([2 * math.pi * 3.25] * 8 + [-math.pi / 2] * 8, device="cpu")
    for w, t in zip(turns(r), [0.25] * 8 + [0.75] * 8):
        assert abs(w / 2 ** 64 - t) < 1e-15


def test_scalings():
    plain = Q.Rotary(64, 10000.0, device="cpu").freqs
    assert plain[0] == 1.0 and plain[31] == pytest.approx(10000.0 ** (-62 / 64), rel=1e-15)
    linear = Q.Rotary(64, 10000.0, scaling="linear", factor=4.0, device="cpu").freqs
    assert all(a == b / 4 for a, b in zip(linear, plain))
    ntk = Q.Rotary(64, 10000.0, scaling="ntk", factor=4.0, device="cpu").freqs
    assert ntk[0] == 1.0 and ntk[31] == pytest.approx(plain[31] / 4, rel=1e-12)  # the ends that the scaling is made for
    y = Q.Rotary(64, 10000.0, scaling="yarn", factor=8.0, original=4096, device="cpu")
    assert y.size == pytest.approx(1 + 0.1 * math.log(8))
    inside = [4096 * f / (2 * math.pi) for f in plain]  # turns within the original context
    for f, g, t in zip(y.freqs, plain, inside):
        if t > 40:
            assert f == g
        elif t < 0.7:
            assert f == pytest.approx(g / 8, rel=1e-12)
        else:
            assert g / 8 <= f <= g
    assert sorted(y.freqs, reverse=True) == y.freqs


# ------------------------------------------------------------------------------------------------- the oracle

def test_oracle_norm():
    y = SO.rms_norm([[3.0, 4.0]], eps=0.0)
    assert np.allclose(y, np.array([[3.0, 4.0]]) / math.sqrt(12.5), rtol=1e-15)
    assert np.allclose(SO.rms_norm([[2.0] * 8], [3.0] * 8, 0.0), 3.0)
    assert np.array_equal(SO.group_scales(np.array([[1.0, -4.0, 2.0, 0.5, 3.0]]), 2.0, 2), [[2.0, 1.0, 1.5]])


def test_oracle_rotation():
    """Lengths of pairs stay, angles add, a quarter turn maps (a, b) to (-b, a)."""
    rng = np.random.default_rng(3)
    x = rng.standard_normal((4, 2, 32))
    f = [0.3 * 0.7 ** j for j in range(8)]
    for pairs in (False, True):
        a = SO.rotate(SO.rotate(x, [2] * 4, f, 1.0, pairs), [5] * 4, f, 1.0, pairs)
        assert np.allclose(a, SO.rotate(x, [7] * 4, f, 1.0, pairs), atol=1e-14)
        assert np.array_equal(a[..., 16:], x[..., 16:])
        q = SO.rotate(x, [1] * 4, [math.pi / 2] * 8, 2.0, pairs)
        u, v = (x[..., 0:16:2], x[..., 1:16:2]) if pairs else (x[..., :8], x[..., 8:16])
        s, t = (q[..., 0:16:2], q[..., 1:16:2]) if pairs else (q[..., :8], q[..., 8:16])
        assert np.allclose(s, -2 * v) and np.allclose(t, 2 * u)


def test_oracle_rotation_is_of_the_difference():
    """A product of two rotated vectors depends on the distance of their positions alone."""
    rng = np.random.default_rng(4)
    q, k = rng.standard_normal((2, 1, 1, 16))
    f = [0.9 ** j for j in range(8)]
    d = [float((SO.rotate(q, [p + 3], f) * SO.rotate(k, [p], f)).sum()) for p in (0, 10, 1000)]
    assert np.allclose(d, d[0], atol=1e-10)


def test_oracle_sampling():
    l = [1.0, 3.0, 2.0, 3.0, -math.inf, math.nan, 0.0]
    assert SO.kept_tokens(l, 1.0)[0] == [1, 3, 2, 0, 6]
    assert SO.kept_tokens(l, 0.0)[0] == [1]
    assert SO.kept_tokens(l, 1.0, top_k=2)[0] == [1, 3] and SO.kept_tokens(l, 1.0, top_k=1)[0] == [1]
    w = np.exp([0.0, 0.0, -1.0, -2.0, -3.0])
    assert SO.kept_tokens(l, 1.0, top_p=(w[:2].sum() + 1e-9) / w.sum())[0] == [1, 3, 2]
    assert SO.kept_tokens(l, 1.0, top_p=(w[:2].sum() - 1e-9) / w.sum())[0] == [1, 3]
    assert SO.kept_tokens(l, 1.0, top_p=0.0)[0] == [1]
    assert SO.kept_tokens(l, 1.0, min_p=math.exp(-1.5))[0] == [1, 3, 2] and SO.kept_tokens(l, 1.0, min_p=2.0)[0] == [1, 3]
    assert SO.kept_tokens(l, 0.5)[1][2] == pytest.approx(math.exp(-2.0))
    assert SO.sample([-math.inf, math.nan], 0.5) == (-1, 0.0)
    # by index: tokens 0 .. 3 of equal weight split [0, 1) evenly
    assert [SO.sample([1.0] * 4, u)[0] for u in (0.0, 0.24, 0.25, 0.5, 0.99)] == [0, 0, 1, 2, 3]
    # frequencies over a grid of u are the probabilities
    us = (np.arange(4000) + 0.5) / 4000
    got = np.bincount([SO.sample(l, float(u))[0] for u in us], minlength=7) / 4000
    assert np.allclose(got[[1, 3, 2, 0, 6]], w / w.sum(), atol=1e-3) and got[4] == got[5] == 0
