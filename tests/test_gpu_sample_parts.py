"""Sampling by parts of a row (vocabularies past 65,536, or few rows of more than 16,384): the same edges as by one
workgroup a row, with special values in single parts, in whole parts and in all of them; and rows that do not depend on
the route that the call's other rows choose."""
from __future__ import annotations

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_sample import SETTINGS, compare, draws, logits_of  # noqa: E402
import bit_weight_only_packed_amd as Q  # noqa: E402

INF, NAN = float("inf"), float("nan")
VOCAB = 70003  # 34 parts of 2,064 tokens and one of less


@pytest.fixture(scope="module", autouse=True)
def _gpu_present():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


@pytest.mark.parametrize("dtype", ["f16", "f32"])
@pytest.mark.parametrize("settings", [dict(), dict(top_k=3), dict(top_p=0.6), dict(temperature=0.0), dict(min_p=0.1),
                                      dict(top_k=40, top_p=0.9, min_p=0.1), dict(top_k=5000, top_p=0.99)])
def test_infinities_and_nan(dtype, settings):
    x = logits_of(14, VOCAB, dtype, 2)
    x[0, 3:40000] = -INF          # whole parts of nothing
    x[1, :] = -INF
    x[2, :] = NAN
    x[3, 7], x[3, 66000] = NAN, NAN
    x[4, 11000], x[4, 30000], x[4, VOCAB - 1] = INF, INF, INF
    x[5, :] = -INF
    x[5, 50001] = 1.5             # one token
    x[6, :20000] = NAN
    x[7, :] = torch.finfo(x.dtype).min
    x[8, 5] = torch.finfo(x.dtype).max
    x[9, :VOCAB - 1] = -INF       # the last
    x[10, 1:] = NAN               # the first
    x[11, 30000:] = torch.finfo(x.dtype).min
    x[12, ::2] = -INF
    for seed in range(2):
        t = compare(x, draws(14, seed), **settings)
        assert int(t[1]) == int(t[2]) == -1 and int(t[5]) == 50001 and int(t[9]) == VOCAB - 1 and int(t[10]) == 0


def test_zero_and_minus_zero_are_equal():
    x = torch.zeros((1, VOCAB)).cuda()
    x[0, ::2] = -0.0
    assert int(Q.sample(x, torch.zeros(1).cuda(), temperature=0.0)) == 0
    for u in (0.1, 0.4, 0.9):
        compare(x, torch.tensor([u]).cuda(), 1.0, 3)
        compare(x, torch.tensor([u]).cuda(), 1.0, 30001)


def test_uniform_numbers_at_their_ends():
    x = torch.zeros((6, VOCAB)).cuda()
    u = torch.tensor([0.0, 1 - 2.0 ** -24, 1.0, 5.0, -3.0, NAN]).cuda()
    assert Q.sample(x, u).tolist() == [0, VOCAB - 1, VOCAB - 1, VOCAB - 1, 0, 0]
    assert Q.sample(x, u, top_k=10).tolist() == [0, 9, 9, 9, 0, 0]
    assert Q.sample(x, u, top_k=50000).tolist() == [0, 49999, 49999, 49999, 0, 0]


def test_odd_parameters_of_rows():
    x = logits_of(8, VOCAB, "f32", 4)
    u = draws(8, 4)
    t = lambda *v: torch.tensor(v, dtype=torch.float32).cuda()  # noqa: E731
    free = Q.sample(x, u)
    assert torch.equal(Q.sample(x, u, top_p=t(*[NAN] * 8)), free)
    assert torch.equal(Q.sample(x, u, min_p=t(*[NAN, -1.0] * 4)), free)
    assert torch.equal(Q.sample(x, u, top_k=torch.full((8,), -5, dtype=torch.int32).cuda()), free)
    first = x.argmax(-1).int()
    assert torch.equal(Q.sample(x, u, temperature=t(*[NAN, -1.0, 0.0, -INF] * 2)), first)
    assert torch.equal(Q.sample(x, u, temperature=t(*[NAN, -1.0, 0.0, -INF] * 2), top_k=7, top_p=0.5), first)
    assert torch.equal(Q.sample(x, u, top_p=-1.0), first) and torch.equal(Q.sample(x, u, top_k=1), first)
    compare(x, u, INF)
    compare(x, u, INF, 40001, 0.5)
    compare(x, u, 1e-30)


@pytest.mark.parametrize("settings", range(len(SETTINGS)))
@pytest.mark.parametrize("kind", ["f16", "f32", "equal"])
def test_rows_do_not_depend_on_the_route(settings, kind):
    """200 rows of 30,011 go by one workgroup each, a few of them by parts: the same tokens and probabilities."""
    n, v = 200, 30011
    if kind == "equal":  # runs of equal logits longer than any list
        x = (torch.randint(0, 3, (n, v), generator=torch.Generator().manual_seed(5)).float() * 0.25).half().cuda()
    else:
        x = logits_of(n, v, kind, 5)
    u = draws(n, settings)
    s = dict(SETTINGS[settings], probs=True)
    t, p = Q.sample(x, u, **s)
    for a, b in ((0, 1), (17, 20), (199, 200)):
        one, q = Q.sample(x[a:b], u[a:b], **s)
        assert torch.equal(one, t[a:b]) and torch.equal(q, p[a:b])


def test_offsets_past_4_gib():
    """Rows that lie farther than 2^32 bytes from the first, at an odd stride."""
    stride, v = (1 << 31) + 7, 20001
    flat = torch.zeros(2 * stride + v, dtype=torch.float16, device="cuda")
    x = flat.as_strided((3, v), (stride, 1))
    x.copy_(logits_of(3, v, "f16", 9))
    u = draws(3, 9)
    for s in (dict(), dict(top_k=50, top_p=0.9)):
        compare(x, u, 0.8, **s)
    many = flat.as_strided((3, 1000), (stride, 1))
    got = Q.sample(many, u, top_k=9)
    assert np.array_equal(got.cpu().numpy(), Q.sample(many.contiguous(), u, top_k=9).cpu().numpy())
