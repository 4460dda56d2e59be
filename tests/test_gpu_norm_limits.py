"""The norm at the ends of its number formats, against the definition in fp64."""
from __future__ import annotations

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from _kv import DT, UNIT, np64  # noqa: E402
from oracle import step_oracle as SO  # noqa: E402
import bit_weight_only_packed_amd as Q  # noqa: E402

CODES = {"int8": (torch.int8, 127.0), "e4m3": (torch.float8_e4m3fn, 448.0)}
TINY = 2.0 ** -149  # fp32's smallest number


@pytest.fixture(scope="module", autouse=True)
def _gpu_present():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


@pytest.mark.parametrize("n", [96, 4096, 20000])
@pytest.mark.parametrize("exp", [-70, -75])
def test_small_elements_beside_large_ones(n, exp):
    """A row whose squares pass fp32 because of one element: the others, 2^140 or more below it, keep the bits that fp32
    has for h / sqrt(mean), and a weight brings them back."""
    g = torch.Generator().manual_seed(n)
    x = (torch.rand((3, n), generator=g, dtype=torch.float64) + 1) * 2.0 ** exp
    x[:, 5] = 2.0 ** 70
    x, w = x.to(torch.bfloat16).cuda(), torch.full((n,), 2.0 ** 60, dtype=torch.bfloat16, device="cuda")
    y = Q.rms_norm(x, w)
    ref = SO.rms_norm(np64(x), np64(w))
    # the output's rounding, the arithmetic of the mean and root, and half of fp32's smallest number times the weight
    assert (np.abs(np64(y) - ref) <= np.abs(ref) * (UNIT["bf16"] + 40 * 2.0 ** -24) + TINY / 2 * 2.0 ** 60).all()


@pytest.mark.parametrize("eps", [2.0 ** -149, 1e-44, 1e-40, 1e-36, 2.0 ** -101, 2.0 ** -99, 1e-20])
@pytest.mark.parametrize("n", [40, 1000, 5120])
def test_squares_too_small_for_fp32(eps, n):
    """Rows of 2^-130 to 2^-40 with an eps no larger than their squares, which fp32 rounds away."""
    g = torch.Generator().manual_seed(n)
    x = torch.randn((19, n), generator=g, dtype=torch.float64) * torch.exp2(torch.arange(-130, -35, 5, dtype=torch.float64))[:, None]
    x[3] = 0
    x = x.to(torch.bfloat16).cuda()
    ref = SO.rms_norm(np64(x), eps=float(np.float32(eps)))
    y = np64(Q.rms_norm(x, eps=eps))
    # the output's rounding, the arithmetic of the sum, root and products, half of bf16's smallest number
    assert (np.abs(y - ref) <= np.abs(ref) * (UNIT["bf16"] + 40 * 2.0 ** -24) + 2.0 ** -134).all()


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("low", [0, 3])
def test_codes_whose_scale_has_few_bits(kind, low):
    """A row with one large element and a group near 2^-140 (sqrt(96) 2^-70 times 8 m, 780 to 7,800 of the smallest
    numbers, or an eighth of that): max / top is a handful of them, and y / scale may pass the type's largest, where
    the code stays at it and keeps its sign."""
    code, top = CODES[kind]
    m = torch.arange(20, 200, 0.5, dtype=torch.float64) * 2.0 ** (-80 - low)
    x = torch.zeros((m.numel(), 96), dtype=torch.float64)
    x[:, 0] = 2.0 ** 70
    x[:, 32], x[:, 33], x[:, 34], x[:, 40] = m * 8, -m * 8, m, -m * 4
    x[:, 64], x[:, 65] = m * 32, -m * 32
    x = x.to(torch.bfloat16).cuda()
    codes, scales = Q.rms_norm(x, quant=code, group=32)
    y = SO.rms_norm(np64(x))
    c, s = np64(codes.float()), np64(scales)
    assert (s[:, 1] < 8 * TINY).any() and (s[:, 1] > 0).any()
    want = SO.group_scales(y, top, 32)
    # y is fp32's, a product of roundings of 2^-23 of it and then to a multiple of 2^-149; so is the scale
    assert (np.abs(s - want) <= want * 2.0 ** -21 + 1.5 * TINY).all()
    wide = np.repeat(s, 32, 1)
    step = 1.0 if kind == "int8" else np.exp2(np.maximum(np.floor(np.log2(np.maximum(np.abs(c), 2.0 ** -6))), -6) - 3)
    held = np.clip(y, -top * wide, top * wide)
    keep = wide > 0
    assert (np.abs(c) <= top).all() and (c[~keep] == 0).all()
    assert (np.abs(c * wide - held) <= wide * step / 2 * (1 + 2.0 ** -10) + np.abs(y) * 2.0 ** -20 + TINY)[keep].all()
    big = keep & (np.abs(y) > 40 * TINY) & (np.abs(y) > wide)
    assert big.any() and (np.sign(c) == np.sign(y))[big].all()


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("group", [32, 128])
def test_codes_are_the_quotients_nearest(kind, dtype, group):
    """Rows of ones have a norm of exactly 1 and y = weight, so every code is known: fp32's max / top and y / scale, rounded
    to nearest even, ties among them (multiples of half a step of a largest value that the type's divides)."""
    code, top = CODES[kind]
    n = 32768
    x = torch.ones((1, n), dtype=DT[dtype], device="cuda")
    for seed in range(24):
        g = torch.Generator().manual_seed(seed)
        w = torch.randn(n, generator=g)
        if seed % 2:  # multiples of 1 / 2 in groups whose largest is 127 / 2 (or 448 / 7) times a small whole number
            m = torch.randint(1, 8, (n // group, 1), generator=g)
            big = m * (63.5 if kind == "int8" else 64.0)
            w = (torch.randint(-120, 121, (n // group, group), generator=g) * m / 4).clamp(-big, big)
            w[:, :1] = big
            w = w.reshape(-1)
        w = w.to(DT[dtype])
        codes, scales = Q.rms_norm(x, w.cuda(), eps=1e-30, quant=code, group=group)
        y = w.float().reshape(-1, group)
        s = y.abs().amax(1, keepdim=True) / torch.tensor(top)
        assert torch.equal(scales.cpu().reshape(-1, 1), s)
        want = y / s
        want = torch.round(want).to(torch.int8) if kind == "int8" else want.to(code)
        assert torch.equal(codes.cpu().float(), want.reshape(1, n).float()), seed
