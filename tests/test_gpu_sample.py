"""GPU tests of dg_sample_logits against its definition in 64 bits."""
import math
import random

import pytest
import torch

import block_diffusion_decoding_gb300 as dg
from tests._paged import DEV

pytestmark = pytest.mark.gpu


# weights are off by 2^-28 of themselves at most and sums by 2^-43 a token: a cumulated weight by 2^-27 of the whole
EPS = 2.0 ** -27


def reference(x, T, k, p, low, u):
    """The definition for one row: (token, logprob, others); others: what it may be as well where u or top-p's border
    is within EPS of the whole weight of another answer."""
    x = x.double()
    x = torch.where(torch.isnan(x), torch.full_like(x, -math.inf), x)
    order = torch.argsort(x, descending=True, stable=True)
    m = x[order[0]]
    if m == -math.inf:
        return -1, -math.inf, ()
    if not T > 0 or k == 1 or p <= 0:
        return order[0].item(), 0.0, ()
    T = min(max(T, 2.0 ** -100), 2.0 ** 100)
    order = order[x[order] > -math.inf]
    w = (x[order] == m).double() if m == math.inf else torch.exp((x[order] - m) / T)
    order, w = order[w > 0], w[w > 0]
    if k > 0:
        order, w = order[:k], w[:k]
    before, all_w = w.cumsum(0) - w, w.sum()

    def draw(p, u):
        o, v = order, w
        if p < 1:
            stay = before < p * all_w
            stay[0] = True
            o, v = o[stay], v[stay]
        if low > 0:
            stay = v >= min(low, 1.0)
            o, v = o[stay], v[stay]
        o, at = torch.sort(o)
        v = v[at]
        mass = v.cumsum(0)
        i = min(int((mass <= min(max(u, 0.0), 1.0) * mass[-1]).sum()), v.numel() - 1)
        return o, i, math.log(v[i] / mass[-1])

    o, i, lp = draw(p, u)
    others = set()
    for q in (p - EPS, p, p + EPS) if p < 1 else (p,):
        o2, first, _ = draw(q, max(u - EPS, 0.0))
        last = draw(q, u + EPS)[1]
        others.update(o2[first:last + 1].tolist())
    return o[i].item(), lp, others


def check(x, T=None, k=None, p=None, low=None, u=None, exact=False):
    """exact: the answer is a matter of whole numbers, and no other is taken."""
    R, V = x.shape
    u = torch.rand(R, generator=torch.Generator().manual_seed(R * V)) if u is None else u
    dev = lambda t, dt: None if t is None else torch.as_tensor(t).to(dt).to(DEV)  # noqa: E731
    xd = x if x.is_cuda else x.to(DEV)
    token = torch.full((R,), -9, dtype=torch.int32, device=DEV)
    logprob = torch.full((R,), 5.0, device=DEV)
    args = dict(temperature=dev(T, torch.float32), top_k=dev(k, torch.int32), top_p=dev(p, torch.float32),
                min_p=dev(low, torch.float32))
    dg.sample_logits(xd, token, dev(u, torch.float32), logprob=logprob, **args)
    at = lambda t, r, off: off if t is None else torch.as_tensor(t).float()[r].item()  # noqa: E731
    for r in range(R):
        want, lp, others = reference(x[r].cpu(), at(T, r, 1.0), int(at(k, r, 0)), at(p, r, 1.0), at(low, r, 0.0),
                                     at(u, r, 0.0))
        if token[r].item() != want:
            assert not exact and token[r].item() in others, (r, token[r].item(), want)
            continue
        got = logprob[r].item()
        # its own rounding, and ln of sums that are off by EPS
        assert got == lp or abs(got - lp) <= 2 ** -24 * abs(lp) + 2 * EPS, (r, got, lp)
    again = torch.full((R,), -9, dtype=torch.int32, device=DEV)
    dg.sample_logits(xd, again, dev(u, torch.float32), **args)      # without logprob
    assert torch.equal(again, token)
    return token


def logits(R, V, seed, dtype, spread=3.0):
    g = torch.Generator().manual_seed(seed)
    return (spread * torch.randn(R, V, generator=g)).to(dtype)


def params(R, seed, T=True, k=True, p=True, low=True):
    r = random.Random(seed)
    return dict(T=[r.choice([0.0, 0.3, 0.7, 1.0, 1.5]) for _ in range(R)] if T else None,
                k=[r.choice([0, 1, 2, 7, 50, 400]) for _ in range(R)] if k else None,
                p=[r.choice([1.0, 0.0, 0.3, 0.9, 0.99]) for _ in range(R)] if p else None,
                low=[r.choice([0.0, 0.01, 0.2, 1.0]) for _ in range(R)] if low else None)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("R,V", [(1, 1), (3, 2), (5, 7), (9, 8), (4, 100), (17, 1001), (6, 4096), (40, 5003),
                                 (3, 32768), (2, 50257), (160, 2049)])
def test_sizes(R, V, dtype):
    x = logits(R, V, R + V, dtype)
    check(x)
    check(x, **params(R, V))
    check(x, **params(R, V + 1, k=False, low=False))
    check(x, **params(R, V + 2, p=False))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("V", [151643, 262144, 393216])
def test_whole_vocabularies(V, dtype):
    for seed in range(3):
        x = logits(6, V, seed, dtype, spread=[0.5, 2.0, 4.0][seed])
        check(x, T=[1.0] * 6)
        check(x, T=[0.8] * 6, k=[0, 50, 1000, 0, 50, 200000], p=[0.9, 0.9, 1.0, 0.5, 1.0, 0.999], low=[0, 0, 0, 0.05, 0.1, 0])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_strided_rows(dtype):
    wide = logits(7, 3000, 1, dtype).to(DEV)
    for V, first in ((2049, 0), (2999, 0), (1, 0), (2048, 8)):
        x = wide[:, first:first + V]
        check(x, **params(7, V))
    check(wide[:, :1500][::2], **params(4, 3))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_equal_logits_are_drawn_exactly(dtype):
    """A flat row: token floor(u V), the border cases included; top-k and top-p keep the lowest indices."""
    V = 4096
    x = torch.full((64, V), -3.25, dtype=dtype)
    u = torch.arange(64) / 64.0
    assert check(x, u=u, exact=True).tolist() == [64 * i for i in range(64)]
    check(x, u=u, p=[0.5] * 64, exact=True)
    check(x, u=u, k=[100] * 64, exact=True)
    check(x, u=u, k=[128] * 64, p=[0.25] * 64, exact=True)
    check(x, u=u, low=[1.0] * 64, exact=True)
    # two levels, masked tokens between
    x[:, ::2] = -math.inf
    check(x, u=u, p=[0.5] * 64, exact=True)
    x[:, 1::4] = 100.0
    check(x, u=u, k=[1025] * 64, p=[0.75] * 64, exact=True)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_masked_infinite_and_nan_logits(dtype):
    V = 5000
    x = logits(12, V, 3, dtype)
    x[0] = -math.inf
    x[1] = NAN = float("nan")
    x[2, ::3] = -math.inf
    x[3, 5:] = -math.inf
    x[4, 1:] = -math.inf
    x[5, [7, 99, 4000]] = math.inf
    x[6, [7, 99, 4000]] = math.inf
    x[7, 100:4000] = NAN
    x[8] = torch.finfo(dtype).min
    x[9, 17:] = torch.finfo(dtype).min
    x[10, 3] = torch.finfo(dtype).max
    x[11, ::2] = -math.inf
    x[11, 1::4] = NAN
    u = torch.full((12,), 0.61)
    check(x, u=u, exact=True)
    check(x, u=u, k=[3] * 12, exact=True)
    check(x, u=u, k=[2] * 12, p=[0.9] * 12, exact=True)
    check(x, u=u, p=[0.4] * 12, low=[0.01] * 12)
    check(x, u=u, T=[0.0] * 12, exact=True)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_extreme_temperatures_and_logits(dtype):
    x = logits(10, 3001, 5, dtype)
    x[5:] *= 1000
    T = [1e-30, 1e-4, 1e-2, 1e4, 1e30, 1e-6, 1.0, 300.0, 1e10, float("inf")]
    check(x, T=T)
    check(x, T=T, p=[0.7] * 10)
    check(x, T=T, k=[40] * 10)
    check(x * 0, T=T)
    x = x.double().abs().mul(-1).sub(1e5).to(dtype)      # all negative, far from zero
    check(x, T=[1.0, 0.1, 10.0, 1e3, 1e-3] * 2)
    check(x, T=[-1.0, float("nan"), 0.0, -0.0, 1.0] * 2, exact=True)


def test_random_numbers_at_the_ends():
    """u = 0: the first kept token, however light; next to 1 and past it: the last that counts."""
    x = logits(4, 3000, 7, torch.float32, spread=6.0)
    check(x, u=torch.zeros(4), exact=True)
    got = check(x, u=torch.zeros(4), T=[0.3] * 4, k=[30] * 4, exact=True)
    for r in range(4):
        assert got[r].item() == min(torch.topk(x[r], 30).indices.tolist())
    one = torch.full((4,), 1.0 - 2.0 ** -24)
    check(x, u=one)
    last = check(x, u=torch.full((4,), 1.0), k=[30] * 4, exact=True)
    for r in range(4):
        assert last[r].item() == max(torch.topk(x[r], 30).indices.tolist())
    dg.sample_logits(x.to(DEV), torch.zeros(4, dtype=torch.int32, device=DEV), torch.full((4,), float("nan"), device=DEV))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_nearby_values(dtype):
    """Cuts between logits that differ in their last bits, or around zero, where such bits are small."""
    g = torch.Generator().manual_seed(1)
    base = torch.randn(6, 6000, generator=g) * torch.tensor([1e-6, 1e-3, 1.0, 1e-30, 30.0, 1e-38])[:, None]
    x = (base + torch.tensor([12.0, 0.0, 0.0, 0.0, -100.0, 0.0])[:, None]).to(dtype)
    for k in (2, 10, 999, 5999):
        check(x, k=[k] * 6)
        check(x, k=[k] * 6, p=[0.5] * 6)
    check(x, p=[0.5] * 6, exact=False)
    check(x, p=[0.9999] * 6)


def test_many_rows_and_repeats():
    """More rows than clusters fit at once; the same inputs give the same tokens; a graph replays."""
    x = logits(3000, 1000, 2, torch.bfloat16).to(DEV)
    u = torch.rand(3000, generator=torch.Generator().manual_seed(0)).to(DEV)
    k = torch.full((3000,), 40, dtype=torch.int32, device=DEV)
    token, again = (torch.zeros(3000, dtype=torch.int32, device=DEV) for _ in range(2))
    dg.sample_logits(x, token, u, top_k=k)
    graph = torch.cuda.CUDAGraph()
    stream = torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=stream):
        dg.sample_logits(x, again, u, top_k=k)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(token, again)
    u.copy_(torch.rand(3000, generator=torch.Generator().manual_seed(1)))
    graph.replay()
    torch.cuda.synchronize()
    assert not torch.equal(token, again)
    dg.sample_logits(x[:0], token[:0], u[:0])


def test_frequencies_follow_the_weights():
    """u over an even grid: every token as often as its weight says, to one."""
    x = torch.tensor([[0.0, 1.0, -math.inf, 2.0, 0.5, -1.0]]).expand(10000, 6).contiguous()
    u = (torch.arange(10000) + 0.5) / 10000
    token = torch.zeros(10000, dtype=torch.int32, device=DEV)
    dg.sample_logits(x.to(DEV), token, u.to(DEV))
    w = torch.softmax(x[0].double(), 0)
    n = torch.bincount(token.cpu().long(), minlength=6)
    assert (n - 10000 * w).abs().max() <= 1


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("ctas", ["1", "2", "8", "16"])
def test_ways_and_clusters(monkeypatch, ctas, dtype):
    """Every way to a token on clusters of every kind: nuclei from a few tokens to nearly all, in logits that lie so
    close that bins of bins hold too many; lists about as long as a CTA has threads, and as they may be."""
    monkeypatch.setenv("DG_SAMPLE_CTAS", ctas)
    V = 60007
    for spread in (0.001, 0.03, 0.3, 1.0, 3.0, 12.0):
        x = logits(5, V, int(spread * 1000), dtype, spread=spread)
        check(x, T=[1.0, 0.9, 1.1, 1.0, 0.5], p=[0.1, 0.5, 0.9, 0.999, 0.7])
        check(x, p=[0.9, 0.5, 1.0, 0.1, 0.9], low=[0.2, 0.0, 0.5, 0.9, 0.01])
    x = logits(7, V, 1, dtype)
    for k in ([254, 255, 256, 257, 258, 300, 2], [1000, 1023, 1024, 1025, 1500, 30000, 60006]):
        check(x, k=k)
        check(x, k=k, p=[0.3, 0.9, 0.95, 0.5, 1.0, 0.8, 0.6], low=[0, 0.01, 0, 0.001, 0.1, 0, 0])
    check(x, T=[1.0, 0.5, 2.0, 1.0, 0.7, 1.5, 1.0])


def test_logprob_far_from_the_largest():
    """A token's log probability where it is large, at temperatures of every size, and where x - m leaves fp32."""
    V = 40
    x = torch.zeros(8, V)
    x[:, 0] = torch.tensor([30.0, -30.0, 1e4, -1e4, 3e38, 1e-3, 5.0, 2.0 ** 20])
    x[:, 1:] = x[:, :1] - torch.tensor([20.0, 25.0, 0.0, 1e-2, 0.0, 1e-30, 3.0, 16.0])[:, None]
    T = [1.0, 1.5, 1e-2, 1e-3, 1e30, 1e-28, 0.25, 1.0]
    for u in (0.0, 0.25, 0.999, 1.0 - 2.0 ** -24):
        check(x, T=T, u=torch.full((8,), u))
    y = x.clone()
    y[:, 1:] = torch.tensor([-3e38] * 8)[:, None]        # whose weight is nothing beside the first's
    check(y, T=T, u=torch.full((8,), 0.5), exact=True)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("value", [-1e4, -1e9, "min", -math.inf])
@pytest.mark.parametrize("first,last", [(300, 20000), (0, 19000), (7000, 19900)])
def test_masks_of_finite_values(dtype, value, first, last):
    """Tokens ruled out by a large negative number or the type's lowest: fewer left than top-k asks for, all of them in
    a few threads' groups; where the temperature lets such a token weigh something, it counts."""
    x = logits(8, 20000, 3, dtype)
    x[:, first:last] = torch.finfo(dtype).min if value == "min" else value
    k = [1, 5, 250, 400, 1000, 1024, 19999, 120]
    for T in (0.05, 1.0, 10.0, 50.0):
        for u in (0.0, 0.3, 0.999):
            check(x, T=[T] * 8, k=k, u=torch.full((8,), u))
        check(x, T=[T] * 8, k=k, p=[0.9] * 8, low=[0.0, 0.01] * 4)
        check(x, T=[T] * 8, p=[0.3, 0.9, 0.999, 1.0] * 2)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_logprob_of_a_token_that_is_nearly_all(dtype):
    """0 for a token that is kept alone, by whichever filter; else off by its own rounding, the others' weights' (2^-28 of
    themselves, which is the result's size) and what all 41 are cut off by, each by up to 2^-43: 41 x 2^-43 < 2^-37."""
    for V in (1, 50, 3001, 151643):
        x = logits(6, V, 3, dtype)
        u = torch.full((6,), 0.7, device=DEV)
        token, logprob = torch.zeros(6, dtype=torch.int32, device=DEV), torch.full((6,), 5.0, device=DEV)
        t, p, low = (torch.full((6,), v, device=DEV) for v in (1e-4, 1e-6, 1.0))
        k = torch.full((6,), 300, dtype=torch.int32, device=DEV)
        x[torch.arange(6), torch.arange(6) * (V // 7)] = 20.0           # one that leads (bf16 has ties)
        xd = x.to(DEV)
        for args in (dict(temperature=t), dict(top_p=p), dict(top_p=p, top_k=k), dict(min_p=low), dict(temperature=t, top_k=k),
                     dict(min_p=low, top_p=p)):
            dg.sample_logits(xd, token, u, logprob=logprob.fill_(5.0), **args)
            assert (logprob == 0).all() and token.tolist() == [r * (V // 7) for r in range(6)], (V, list(args))
    x = torch.full((16, 41), -math.inf)
    x[:, 0] = 0.0
    for r in range(16):
        x[r, 1:] = -3.0 - 1.5 * r
    x = x.to(dtype)
    u = torch.zeros(16, device=DEV)
    token, logprob = torch.ones(16, dtype=torch.int32, device=DEV), torch.zeros(16, device=DEV)
    for args in (dict(), dict(top_k=torch.full((16,), 40, dtype=torch.int32, device=DEV))):
        dg.sample_logits(x.to(DEV), token, u, logprob=logprob, **args)
        n = 39 if args else 40
        want = -torch.log1p(n * torch.exp(x[:, 1].double()))
        assert (token == 0).all()
        assert ((logprob.cpu().double() - want).abs() <= want.abs() * 2 ** -21 + 2 ** -37 + 2 ** -26 * (want < -0.06)).all(), (logprob, want)
