"""Sampling against its definition in fp64: tokens equal, probabilities to fp32."""
from __future__ import annotations

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from oracle import step_oracle as SO  # noqa: E402
import bit_weight_only_packed_amd as Q  # noqa: E402

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module", autouse=True)
def _gpu_present():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def compare(logits, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """Every row's token is the definition's.  prob: weights are off by 2^-44 of the largest, at most 2^20 of them
    in the sum; then a rounding to fp32."""
    tokens, probs = Q.sample(logits, u, temperature=temperature, top_k=top_k, top_p=top_p, min_p=min_p, probs=True)
    def row(v, i):
        return float(np.float32(v[i].item())) if torch.is_tensor(v) else float(np.float32(v))
    l = logits.double().cpu().numpy()
    for i in range(l.shape[0]):
        want, p = SO.sample(l[i], row(u, i), row(temperature, i), int(row(top_k, i)), row(top_p, i), row(min_p, i))
        assert int(tokens[i]) == want, (i, int(tokens[i]), want)
        assert abs(float(probs[i]) - p) <= 2.0 ** -23 * p + 2.0 ** -40, i
    return tokens


def draws(n, seed):
    return torch.rand((n,), generator=torch.Generator().manual_seed(seed)).cuda()


def logits_of(rows, vocab, dtype, seed, scale=2.2):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((rows, vocab), generator=g) * scale
    x.scatter_add_(1, torch.randint(0, vocab, (rows, 8), generator=g), torch.rand((rows, 8), generator=g) * 8)
    return x.to(TYPES[dtype]).cuda()


SETTINGS = [dict(), dict(temperature=0.7), dict(top_k=1), dict(top_k=5), dict(top_k=50, temperature=1.3), dict(top_p=0.9),
            dict(top_p=0.3, temperature=0.5), dict(min_p=0.1), dict(top_k=40, top_p=0.95, min_p=0.02, temperature=0.8),
            dict(temperature=0.0), dict(top_p=0.0), dict(top_p=0.999, temperature=2.0), dict(top_k=10 ** 6),
            dict(temperature=50.0, top_p=0.5), dict(temperature=0.01, top_k=3), dict(top_k=700, top_p=0.6, temperature=3.0)]


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("rows,vocab", [(1, 1), (2, 2), (3, 7), (2, 8), (4, 1000), (3, 2049), (2, 5003), (2, 17001)])
@pytest.mark.parametrize("settings", range(len(SETTINGS)))
def test_against_the_definition(dtype, rows, vocab, settings):
    compare(logits_of(rows, vocab, dtype, rows * vocab + settings), draws(rows, settings), **SETTINGS[settings])


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("vocab", [131071, 65536])
def test_large_vocabularies(dtype, vocab):
    n = len(SETTINGS)
    x = logits_of(n, vocab, dtype, vocab)
    get = lambda k, d: torch.tensor([s.get(k, d) for s in SETTINGS])  # noqa: E731
    compare(x, draws(n, 3), get("temperature", 1.0).float().cuda(), get("top_k", 0).int().cuda(),
            get("top_p", 1.0).float().cuda(), get("min_p", 0.0).float().cuda())


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("top_k", [900, 1024, 1025, 2048, 3000, 20000, 65000])
@pytest.mark.parametrize("top_p", [1.0, 0.999, 0.7, 0.1])
def test_large_counts_with_shares(dtype, top_k, top_p):
    """Kept tokens by the thousand: the last of them is found among those of one bucket, of two, or of a few."""
    x = logits_of(3, 66000, dtype, top_k, 1.2)
    heat = torch.tensor([1.0, 4.0, 0.4]).cuda()
    compare(x, draws(3, top_k), heat, top_k, top_p)
    compare(x, draws(3, top_k + 1), heat, 0, top_p, 0.001)


@pytest.mark.parametrize("vocab", [600, 3000, 20000])
@pytest.mark.parametrize("levels", [1, 2, 5, 40])
def test_equal_logits(vocab, levels):
    """Cuts among equal logits go by index, in runs longer than any list of them."""
    g = torch.Generator().manual_seed(levels)
    x = (torch.randint(0, levels, (6, vocab), generator=g).float() * 0.25).half().cuda()
    u = draws(6, levels)
    for k in (1, 3, vocab // 3, vocab - 1, vocab):
        compare(x, u, 1.0, k)
    for p in (0.001, 0.25, 0.5, 0.999):
        compare(x, u, 1.0, 0, p)
        compare(x, u, 0.5, vocab // 2, p)
    compare(x, u, 1.0, vocab // 2, 0.5, 0.9)


def test_fp32_logits_closer_than_any_step():
    """Neighbouring fp32 numbers: thousands of distinct logits in one bucket."""
    base = torch.arange(9000, dtype=torch.int32)
    x = (base[torch.randperm(9000, generator=torch.Generator().manual_seed(1))] + 0x40000000).view(torch.float32)[None].cuda()
    for k in (1, 2, 1000, 4321, 8999):
        compare(x, draws(1, k), 1.0, k)
    compare(x, draws(1, 5), 1.0, 0, 0.37)
    compare(x, draws(1, 6), 1e-6, 4000, 0.9)


def test_infinities_and_nan():
    x = torch.randn((9, 50), generator=torch.Generator().manual_seed(2)).cuda()
    x[0, 3:40] = -INF
    x[1, :] = -INF
    x[2, :] = NAN
    x[3, 7], x[3, 9] = NAN, NAN
    x[4, 11], x[4, 30] = INF, INF
    x[5, 1:] = -INF
    x[6, 0] = NAN
    x[7, :] = torch.finfo(torch.float32).min
    x[8, 5] = 3e38
    for s in (dict(), dict(top_k=3), dict(top_p=0.6), dict(temperature=0.0), dict(top_k=40, top_p=0.9, min_p=0.1)):
        for seed in range(3):
            t = compare(x, draws(9, seed), **s)
            assert int(t[1]) == int(t[2]) == -1


def test_zero_and_minus_zero_are_equal():
    x = torch.tensor([[-0.0, 0.0, -0.0, 0.0]]).cuda()
    assert int(Q.sample(x, torch.zeros(1).cuda(), temperature=0.0)) == 0
    for u in (0.1, 0.4, 0.6, 0.9):
        compare(x, torch.tensor([u]).cuda(), 1.0, 3)


def test_uniform_numbers_at_their_ends():
    """0 takes the first kept token, the largest below 1 the last; what lies outside is held to them."""
    x = torch.zeros((6, 100)).cuda()
    u = torch.tensor([0.0, 1 - 2.0 ** -24, 1.0, 5.0, -3.0, NAN]).cuda()
    assert Q.sample(x, u).tolist() == [0, 99, 99, 99, 0, 0]
    assert Q.sample(x, u, top_k=10).tolist() == [0, 9, 9, 9, 0, 0]


def test_odd_parameters_of_rows():
    """NaN: no limit (of temperature: the first token); negative counts and shares."""
    x = logits_of(8, 300, "f32", 4)
    u = draws(8, 4)
    t = lambda *v: torch.tensor(v, dtype=torch.float32).cuda()  # noqa: E731
    free = Q.sample(x, u)
    assert torch.equal(Q.sample(x, u, top_p=t(*[NAN] * 8)), free)
    assert torch.equal(Q.sample(x, u, min_p=t(*[NAN, -1.0] * 4)), free)
    assert torch.equal(Q.sample(x, u, top_k=torch.full((8,), -5, dtype=torch.int32).cuda()), free)
    first = x.argmax(-1).int()
    assert torch.equal(Q.sample(x, u, temperature=t(*[NAN, -1.0, 0.0, -INF] * 2)), first)
    assert torch.equal(Q.sample(x, u, top_p=-1.0), first) and torch.equal(Q.sample(x, u, top_k=1), first)
    compare(x, u, INF)  # all tokens alike
    compare(x, u, 1e-30)


def test_frequencies():
    """4,096 evenly spaced numbers: every token comes as often as its probability says, to one."""
    x = logits_of(1, 60, "f16", 9, 1.0)
    n = 4096
    got = torch.bincount(Q.sample(x.expand(n, 60), (torch.arange(n) + 0.5).div(n).cuda(), top_k=30, top_p=0.9).long(), minlength=60)
    order, w = SO.kept_tokens(x[0].double().cpu().numpy(), 1.0, 30, 0.9)
    want = np.zeros(60)
    want[order] = w / w.sum() * n
    assert (np.abs(got.cpu().numpy() - want) <= 1.0 + 1e-6).all()


def test_strides_and_alignment():
    big = logits_of(5, 4001, "bf16", 3)
    x = big[:, 3:3004]
    u = draws(5, 1)
    assert torch.equal(compare(x, u, 0.9, 20, 0.9), Q.sample(x.contiguous(), u, temperature=0.9, top_k=20, top_p=0.9))
    compare(big[::2, 1:2000], draws(3, 2), 0.9, 0, 0.5)


def test_rows_do_not_depend_on_the_call():
    x, u = logits_of(70, 9001, "f16", 5), draws(70, 5)
    s = dict(temperature=0.9, top_k=300, top_p=0.9, min_p=0.01, probs=True)
    t, p = Q.sample(x, u, **s)
    for i in (0, 33, 69):
        a, b = Q.sample(x[i:i + 1], u[i:i + 1], **s)
        assert torch.equal(a, t[i:i + 1]) and torch.equal(b, p[i:i + 1])


def test_many_rows():
    """More rows than one launch takes."""
    n = 4096 * 2 + 5
    x, u = logits_of(n, 40, "f16", 6), draws(n, 6)
    t = Q.sample(x, u, top_k=9, top_p=0.8)
    for i in (0, 4095, 4096, 8191, 8192, n - 1):
        want, _ = SO.sample(x[i].double().cpu().numpy(), float(u[i]), 1.0, 9, float(np.float32(0.8)))
        assert int(t[i]) == want
    parts = [Q.sample(x[a:a + 1000], u[a:a + 1000], top_k=9, top_p=0.8) for a in range(0, n, 1000)]
    assert torch.equal(torch.cat(parts), t)


def test_many_rows_in_parts():
    """The same where rows go in parts: one row's logits for all of them, a uniform number each."""
    n, v = 4096 + 70, 66001
    x, u = logits_of(1, v, "f16", 8), draws(n, 8)
    t, p = Q.sample(x.expand(n, v), u, temperature=0.8, top_k=40, top_p=0.9, probs=True)
    order, w = SO.kept_tokens(x[0].double().cpu().numpy(), float(np.float32(0.8)), 40, float(np.float32(0.9)))
    by = np.argsort(order)
    run = np.cumsum(w[by])
    pick = by[np.searchsorted(run, u.double().cpu().numpy() * run[-1], side="right")]
    assert np.array_equal(t.cpu().numpy(), np.array(order)[pick])
    assert np.allclose(p.cpu().numpy(), w[pick] / run[-1], rtol=2.0 ** -23, atol=0)


def test_refusals():
    x, u = logits_of(3, 100, "f16", 1), draws(3, 1)
    with pytest.raises(ValueError, match="u must"):
        Q.sample(x, u[:2])
    with pytest.raises(ValueError, match="top_k"):
        Q.sample(x, u, top_k=torch.zeros(3).cuda())
    with pytest.raises(ValueError, match="logits"):
        Q.sample(x.int(), u)
    with pytest.raises(ValueError, match="contiguous"):
        Q.sample(x.t(), draws(100, 1))
    with pytest.raises(ValueError, match="out"):
        Q.sample(x, u, out=torch.zeros(3, dtype=torch.int64).cuda())
    with pytest.raises(Q.QGError, match="workspace"):
        Q.sample(x, u, workspace=torch.zeros(8, dtype=torch.uint8).cuda())
    assert Q.sample(x[:0], u[:0]).shape == (0,)


def test_streams_and_graph_replays():
    x, u = logits_of(6, 30011, "f16", 7), draws(6, 7)
    s = dict(temperature=0.9, top_k=300, top_p=0.9, min_p=0.01)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    want = Q.sample(x, u, **s)
    got = Q.sample(x, u, stream=side, **s)
    side.synchronize()
    assert torch.equal(got, want)
    # two graphs with workspaces of their own, and one that both share in turn
    space = torch.empty(Q.sample_workspace(6, 30011), dtype=torch.uint8, device="cuda")
    outs = [torch.empty(6, dtype=torch.int32, device="cuda") for _ in range(2)]
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    heat = torch.full((6,), 0.9, device="cuda")
    torch.cuda.synchronize()
    for g, o, k in zip(graphs, outs, (300, 0)):
        with torch.cuda.graph(g):
            Q.sample(x, u, temperature=heat, top_k=k, top_p=0.9, out=o, workspace=space)
    for i in range(4):
        x.copy_(logits_of(6, 30011, "f16", 70 + i))
        u.copy_(draws(6, 70 + i))
        heat.fill_(0.5 + 0.2 * i)
        for g in graphs:
            g.replay()
        for o, k in zip(outs, (300, 0)):
            want = Q.sample(x, u, temperature=heat, top_k=k, top_p=0.9)
            torch.cuda.synchronize()
            assert torch.equal(o, want)
