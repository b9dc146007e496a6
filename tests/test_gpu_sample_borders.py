"""GPU tests of dg_sample_logits where its filters' borders lie far down the row, or among tokens that weigh next to
nothing."""
import math

import pytest
import torch

import block_diffusion_decoding_gb300 as dg
from tests._paged import DEV
from tests.test_gpu_sample import check, logits

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("ctas", [None, "1", "16"])
def test_top_k_holds_for_u_of_zero(monkeypatch, ctas, dtype):
    """k above 1024, the k-th token more than 64 factors of 2 below the largest: u = 0 draws the first token of the
    vocabulary among the first k, however light, and none behind them."""
    if ctas is not None:
        monkeypatch.setenv("DG_SAMPLE_CTAS", ctas)
    x = logits(8, 20000, 11, dtype)
    k = [1025, 1100, 1500, 2000, 3000, 4000, 5000, 19999]
    zero = torch.zeros(8)
    for T in (0.02, 0.05, 0.1, 0.3):
        got = check(x, T=[T] * 8, k=k, u=zero, exact=True).tolist()
        for r in range(7):
            assert got[r] in torch.sort(x[r], descending=True, stable=True).indices[:k[r]].tolist(), (T, r)
        check(x, T=[T] * 8, k=k, u=zero, low=[1e-30, 1e-36, 0.0, 1e-20] * 2, exact=True)
        check(x, T=[T] * 8, k=k, u=torch.full((8,), 0.4), p=[0.9, 1.0] * 4)
        check(x, T=[T] * 8, k=k, u=torch.ones(8))
    if dtype is torch.float32:                           # (weights by 64-bit arithmetic)
        check(x + 1e5, T=[0.05] * 8, k=k, u=zero, exact=True)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_top_k_among_more_equal_tokens_than_are_sorted(dtype):
    """The k-th token among thousands of its value, which a list does not hold: the first of them by index are kept."""
    x = logits(8, 20000, 12, dtype, spread=1.5).round()
    k = [1000, 1024, 900, 700, 500, 1023, 2, 1500]
    for T in (0.02, 0.05, 1.0):
        for u in (0.0, 0.5, 1.0):
            check(x, T=[T] * 8, k=k, u=torch.full((8,), u), exact=u == 0.0)


def test_top_p_next_to_one_in_a_long_tail():
    """One token that is nearly all, and hundreds of thousands beside it: 2^-24 of the whole weight are thousands of
    them, and top-p's border lies among them.  The time is bounded too: a border is found by halving, not token by
    token."""
    V, rows = 262144, [(-24, 0.3, 0.999995), (-26, 0.5, 0.999999), (-20, 1.0, 0.99995), (-22, 0.1, 0.99999),
                       (-26, 0.5, 1 - 2.0 ** -24), (-24, 0.3, 0.9999999), (-18, 0.01, 0.999), (-23, 2.0, 0.9999)]
    R = len(rows)
    g = torch.Generator().manual_seed(5)
    x = torch.randn(R, V, generator=g) * torch.tensor([s for _, s, _ in rows])[:, None]
    x += torch.tensor([float(m) for m, _, _ in rows])[:, None]
    x[torch.arange(R), torch.randint(V, (R,), generator=g)] = 0.0
    p = [p for _, _, p in rows]
    for u in (1.0, 1.0 - 2.0 ** -24, 1.0 - 2.0 ** -23, 1.0 - 2.0 ** -21, 0.5, 0.0):
        check(x, p=p, u=torch.full((R,), u))
        check(x, p=p, u=torch.full((R,), u), k=[200000, 0] * 4, low=[0.0, 0.0, 1e-14, 1e-11] * 2)
    check(x.bfloat16(), p=p, u=torch.ones(R))
    xd, token = x.to(DEV), torch.zeros(R, dtype=torch.int32, device=DEV)
    pd, ud = torch.tensor(p, device=DEV), torch.full((R,), 0.5, device=DEV)
    at = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
    for _ in range(2):
        at[0].record()
        dg.sample_logits(xd, token, ud, top_p=pd)
        at[1].record()
    torch.cuda.synchronize()
    assert at[0].elapsed_time(at[1]) < 20.0              # (some 50 passes of 10 us)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_the_split_of_a_row_changes_no_bit(monkeypatch, dtype):
    """Tokens and log probabilities are the same for any number of CTAs a row, and for a row alone and in a batch."""
    V, R = 150001, 12
    x = logits(R, V, 21, dtype)
    x[4:8] = x[4:8] * 0.1 - 30.0                         # one token, and many that weigh next to nothing
    x[4:8, 777] = 1.0
    x[8:10] = -31.0
    x[8:10, 100000] = 0.0
    xd = x.to(DEV)
    f = lambda v: torch.tensor(v, device=DEV)  # noqa: E731
    ways = [dict(), dict(top_p=f([0.9, 0.5, 0.99, 0.9999] * 3)), dict(min_p=f([0.01, 1e-12, 0.0, 1e-5] * 3)),
            dict(top_k=f([50, 1024, 1500, 100000] * 3).int(), top_p=f([0.95] * R))]

    def draw(x, u, args):
        token = torch.full((x.shape[0],), -9, dtype=torch.int32, device=DEV)
        logprob = torch.full((x.shape[0],), 5.0, device=DEV)
        dg.sample_logits(x, token, u, logprob=logprob, **args)
        return token.tolist(), logprob.view(torch.int32).tolist()

    g = torch.Generator().manual_seed(1)
    for way in ways:
        for u in [torch.rand(R, generator=g) for _ in range(4)] + [torch.zeros(R), torch.full((R,), 1 - 2.0 ** -24)]:
            u = u.to(DEV)
            got = []
            for ctas in ("1", "2", "4", "8", "16"):
                monkeypatch.setenv("DG_SAMPLE_CTAS", ctas)
                got.append(draw(xd, u, way))
            monkeypatch.delenv("DG_SAMPLE_CTAS")
            got.append(draw(xd, u, way))
            for r in range(R):
                one = draw(xd[r:r + 1].clone(), u[r:r + 1].clone(), {n: t[r:r + 1].clone() for n, t in way.items()})
                assert (one[0][0], one[1][0]) == (got[0][0][r], got[0][1][r]), (list(way), r)
            assert all(a == got[0] for a in got), list(way)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("V", [262145, 393216])
def test_sums_of_the_longest_rows_hold(V, dtype):
    """Equal logits fill a row's sum to its last bit: token floor(u V) of whole numbers, by every way, at temperatures
    that put the largest weight at either end of its range."""
    R = 6
    x = torch.full((R, V), -3.296875, dtype=dtype)
    T = [0.77, 1.0, 0.3, 3.1, 1.7, 0.9]
    for u in (torch.arange(R) / 8.0 + 2.0 ** -10, torch.full((R,), 1 - 2.0 ** -24), torch.zeros(R)):
        check(x, T=T, u=u, exact=True)
        check(x, T=T, u=u, p=[0.5, 0.75, 0.3, 0.9, 0.99, 0.999969482421875], exact=True)
        check(x, T=T, u=u, k=[1025, 2000, 100000, V - 1, 1, 300000], exact=True)
        check(x, T=T, u=u, k=[1025, 2000, 100000, V - 1, 1, 300000], p=[0.5] * R, low=[0.5] * R, exact=True)
