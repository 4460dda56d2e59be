"""The norm with the residual's addition against its definition in fp64: types, odd sizes and strides, codes with
scales, extreme values, streams and graphs."""
from __future__ import annotations

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from _kv import DT, UNIT, np64, rand  # noqa: E402
from oracle import step_oracle as SO  # noqa: E402
import bit_weight_only_packed_amd as Q  # noqa: E402

EPS32 = 2.0 ** -24
# fp32 arithmetic: a chunk's and the workgroup's sum of squares (at most 32 + 6 + 16 roundings in a row, half of whose
# relative error reaches the root), the mean, the root, the reciprocal (4 roundings of 1 to 2 units) and two products
ARITH = (27 + 8 + 2) * EPS32
CODES = {"int8": (torch.int8, 127.0), "e4m3": (torch.float8_e4m3fn, 448.0)}


@pytest.fixture(scope="module", autouse=True)
def _gpu_present():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def summed(x, res):
    """What stands in the residual: the fp32 sum, rounded once."""
    return x if res is None else (x.float() + res.float()).to(x.dtype)


def check(y, ref, dtype):
    tol = np.abs(ref) * (UNIT[dtype] + ARITH) + 2.0 ** -25  # (half the smallest fp16 number)
    err = np.abs(np64(y) - ref)
    assert (err <= tol).all(), float((err / tol).max())


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("rows,n", [(1, 1), (1, 7), (3, 8), (2, 63), (5, 64), (1, 511), (4, 1280), (1, 5120), (33, 5120),
                                    (2, 8191), (1, 8200), (3, 17408), (1, 32768), (600, 1030), (700, 5120), (1, 32761), (67, 128), (1001, 72), (9, 200), (7, 257)])
@pytest.mark.parametrize("residual,weight", [(True, True), (False, True), (True, False), (False, False)])
def test_against_the_definition(dtype, rows, n, residual, weight):
    x = rand((rows, n), dtype, rows + n)
    res = rand((rows, n), dtype, rows + n + 1, 3.0) if residual else None
    w = rand((n,), dtype, n + 2) if weight else None
    h = summed(x, res)
    y = Q.rms_norm(x, w, residual=res, eps=1e-5)
    if residual:
        assert torch.equal(res, h)
    check(y, SO.rms_norm(np64(h), None if w is None else np64(w), 1e-5), dtype)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("rows,n,group", [(1, 1, 0), (3, 5, 32), (2, 128, 128), (5, 1280, 64), (2, 1000, 32), (4, 1001, 128),
                                          (3, 17408, 128), (2, 17408, 0), (700, 520, 64), (2, 32768, 32), (1, 8191, 0), (65, 128, 0), (67, 40, 128), (33, 72, 64), (5, 250, 32)])
def test_codes(dtype, kind, rows, n, group):
    x, res, w = rand((rows, n), dtype, n), rand((rows, n), dtype, n + 1), rand((n,), dtype, n + 2)
    h = summed(x, res)
    code, top = CODES[kind]
    codes, scales = Q.rms_norm(x, w, residual=res, quant=code, group=group)
    assert torch.equal(res, h) and codes.dtype == code and scales.dtype == torch.float32
    ref = SO.rms_norm(np64(h), np64(w), 1e-6)
    s = np64(scales)
    want = SO.group_scales(ref, top, group)
    assert s.shape == want.shape
    assert (np.abs(s - want) <= want * (ARITH + 2 * EPS32)).all()
    g = group or n
    wide = np.repeat(s, g, 1)[:, :n]
    c = np64(codes.float())
    # half a step (of 1, or of an eighth of the code's power of two, 2^-9 at least), and what y and y / s are off by
    ratio = np.abs(ref) / np.where(wide > 0, wide, 1)
    step = np.ones_like(ratio) if kind == "int8" else np.exp2(np.maximum(np.floor(np.log2(np.maximum(ratio, 2.0 ** -6))), -6) - 3)
    assert (np.abs(c * wide - ref) <= wide * step / 2 * (1 + 2.0 ** -12) + np.abs(ref) * (2 * ARITH + 6 * EPS32)).all()
    assert (np.abs(c) <= top).all()


def test_strides_alignment_and_in_place():
    """Rows inside wider tensors at odd offsets; x normed over itself; neighbours left alone."""
    big, stream = rand((9, 1003), "f16", 1), rand((9, 777), "f16", 2)
    x, res = big[:, 5:505], stream[:, 3:503]
    keep_b, keep_s = big.clone(), stream.clone()
    out = torch.full((9, 601), 7.0, dtype=torch.float16, device="cuda")
    h = summed(x, res)
    Q.rms_norm(x, None, residual=res, out=out[:, 1:501])
    assert torch.equal(res, h) and torch.equal(big, keep_b)
    check(out[:, 1:501], SO.rms_norm(np64(h)), "f16")
    assert (out[:, 0] == 7).all() and (out[:, 501:] == 7).all()
    assert torch.equal(stream[:, :3], keep_s[:, :3]) and torch.equal(stream[:, 503:], keep_s[:, 503:])
    ref = SO.rms_norm(np64(x))
    assert Q.rms_norm(x, out=x).data_ptr() == x.data_ptr()
    check(x, ref, "f16")
    assert torch.equal(big[:, :5], keep_b[:, :5]) and torch.equal(big[:, 505:], keep_b[:, 505:])
    # columns of one tensor: x, residual and out side by side
    t = rand((4, 96), "bf16", 3)
    h = summed(t[:, :32], t[:, 32:64])
    Q.rms_norm(t[:, :32], residual=t[:, 32:64], out=t[:, 64:])
    check(t[:, 64:], SO.rms_norm(np64(h)), "bf16")
    # one row for all (a stride of 0)
    one = rand((1, 40), "f16", 4)
    check(Q.rms_norm(one.expand(3, 40)), np.repeat(SO.rms_norm(np64(one)), 3, 0), "f16")


def test_code_outputs_given():
    x = rand((5, 200), "f16", 5)
    out = torch.zeros((5, 300), dtype=torch.int8, device="cuda")
    scales = torch.zeros((5, 4), device="cuda")
    a, b = Q.rms_norm(x, quant=torch.int8, group=64, out=out[:, 50:250], scales=scales)
    c, s = Q.rms_norm(x, quant=torch.int8, group=64)
    assert torch.equal(a, c) and torch.equal(b, s) and b.data_ptr() == scales.data_ptr()
    assert (out[:, :50] == 0).all() and (out[:, 250:] == 0).all()


def test_large_and_small_values():
    """Squares past fp32's range (bf16), rows of zeros, the smallest fp16 numbers."""
    for exp in (60, 64, 100, 126):
        x = (rand((3, 1030), "bf16", exp).double() * 2.0 ** exp / 8).to(torch.bfloat16)
        check(Q.rms_norm(x, eps=1e-6), SO.rms_norm(np64(x)), "bf16")
    x = torch.zeros((2, 100), dtype=torch.float16, device="cuda")
    assert (Q.rms_norm(x) == 0).all()
    codes, scales = Q.rms_norm(x, quant=torch.float8_e4m3fn, group=32)
    assert (codes.float() == 0).all() and (scales == 0).all()
    x[0] = 2.0 ** -24
    check(Q.rms_norm(x, eps=1e-20), SO.rms_norm(np64(x), eps=float(np.float32(1e-20))), "f16")


def test_non_finite_rows_stay_their_own():
    x = rand((4, 300), "f16", 6)
    x[1, 7], x[2, 250] = float("nan"), float("inf")
    y = Q.rms_norm(x)
    ref = SO.rms_norm(np64(x))
    check(y[[0, 3]], ref[[0, 3]], "f16")
    assert torch.isnan(y[1]).all()
    assert torch.isnan(y[2, 250]) and (y[2, :250] == 0).all()
    codes, scales = Q.rms_norm(x, quant=torch.int8, group=128)
    assert torch.isnan(scales[1]).all() and (codes[1] == 0).all()
    assert torch.isnan(scales[2, 1]) and scales[2, 0] == 0 and (codes[2] == 0).all()
    assert torch.isfinite(scales[[0, 3]]).all()


def test_rows_do_not_depend_on_the_call():
    """A row alone and among few or many has the same bits; so has every repeat."""
    for n in (128, 200, 500, 5120, 17408):
        x, w = rand((2100, n), "f16", 8), rand((n,), "f16", 9)
        y = Q.rms_norm(x, w)
        for i in (0, 17, 2099):
            assert torch.equal(Q.rms_norm(x[i:i + 1], w), y[i:i + 1])
        assert torch.equal(Q.rms_norm(x[:40], w), y[:40]) and torch.equal(Q.rms_norm(x, w), y)


def test_refusals():
    x = rand((3, 64), "f16", 1)
    with pytest.raises(ValueError, match="weight"):
        Q.rms_norm(x, rand((63,), "f16", 1))
    with pytest.raises(ValueError, match="residual"):
        Q.rms_norm(x, residual=rand((3, 64), "bf16", 1))
    with pytest.raises(ValueError, match="contiguous"):
        Q.rms_norm(rand((64, 3), "f16", 1).t())
    with pytest.raises(ValueError, match="quant"):
        Q.rms_norm(x, quant=torch.uint8)
    with pytest.raises(ValueError, match="scales"):
        Q.rms_norm(x, scales=torch.zeros(3, 1, device="cuda"))
    with pytest.raises(Q.QGError, match="overlaps"):
        Q.rms_norm(x, residual=x)
    with pytest.raises(Q.QGError, match="group"):
        Q.rms_norm(x, quant=torch.int8, group=48)
    with pytest.raises(Q.QGError, match="eps"):
        Q.rms_norm(x, eps=0.0)
    assert Q.rms_norm(x[:0]).shape == (0, 64)


def test_streams_and_graph_replays():
    x, w = rand((8, 5120), "f16", 1), rand((5120,), "f16", 2)
    start = rand((8, 5120), "f16", 3)
    res, out = start.clone(), torch.empty_like(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    want = Q.rms_norm(x, w, residual=start.clone())
    got = Q.rms_norm(x, w, residual=res, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    res.copy_(start)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        Q.rms_norm(x, w, residual=res, out=out)
    stand = start.clone()
    res.copy_(start)
    for _ in range(4):
        graph.replay()
        want = Q.rms_norm(x, w, residual=stand)
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(res, stand)
