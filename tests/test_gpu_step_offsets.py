"""Norm and rotation of rows that lie farther than 2^32 bytes apart."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from _kv import rand  # noqa: E402
import bit_weight_only_packed_amd as Q  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _gpu_present():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def far(shape, stride, dtype=torch.float16):
    """Rows of `shape` at a stride of that many elements, and the memory that they lie in."""
    width = torch.Size(shape[1:]).numel()
    flat = torch.zeros((shape[0] - 1) * stride + width, dtype=dtype, device="cuda")
    inner = [torch.Size(shape[i + 1:]).numel() for i in range(1, len(shape))]
    return flat.as_strided(shape, (stride, *inner))


@pytest.mark.parametrize("n", [200, 5120])
def test_norm(n):
    x, res, w = rand((3, n), "f16", 1), rand((3, n), "f16", 2), rand((n,), "f16", 3)
    fx, fr, fo = far((3, n), (1 << 31) + 9), far((3, n), (1 << 31) + 5), far((3, n), (1 << 31) + 3)
    fx.copy_(x)
    fr.copy_(res)
    Q.rms_norm(fx, w, residual=fr, out=fo)
    y = Q.rms_norm(x, w, residual=res)
    assert torch.equal(fo, y) and torch.equal(fr, res)
    codes = far((3, n), (1 << 32) + 3, torch.int8)
    a, s = Q.rms_norm(fx, w, quant=torch.int8, group=64, out=codes)
    b, t = Q.rms_norm(x, w, quant=torch.int8, group=64)
    assert torch.equal(a, b) and torch.equal(s, t)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotate(interleaved):
    x, p = rand((3, 5, 128), "f16", 4), torch.tensor([0, 77, 1 << 20], dtype=torch.int32, device="cuda")
    r = Q.Rotary(64, interleaved=interleaved)
    want = r.rotate(x, p)
    fx, fo = far((3, 5, 128), (1 << 31) + 8), far((3, 5, 128), (1 << 31) + 16)
    fx.copy_(x)
    assert torch.equal(r.rotate(fx, p, out=fo), want)
    assert torch.equal(r.rotate(fx, p, out=fx), want)
    # heads far apart
    hx = far((5, 3, 128), (1 << 31) + 8).transpose(0, 1)
    hx.copy_(x)
    assert torch.equal(r.rotate(hx, p), want)
