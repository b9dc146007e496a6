"""How exact the paged attention's single-CTA kernel is: it multiplies each softmax weight as two bf16 halves, so
its output is off by little more than its own rounding, where one bf16 weight would be off by as much again."""
import pytest
import torch

from tests._paged import Batch, close

# A weight p in fp32 is split into hi, a bf16 less than two of its steps (2^-7 of p at most) below p, and
# lo = bf16(p - hi): p - hi is exact in fp32 and below 2^-6 p, and rounded within 2^-8 of itself, so the halves' sum
# is within 2^-14 p.  Scores below 64 in fp32 and their exponentials: 2^-12, as in tests/_paged.py, which covers
# fp32 sums of up to 1000 products as well (1000 / 16 steps of two halves, each within 2^-23: 2^-16).
WEIGHTS = 2.0 ** -14 + 2.0 ** -12


def batch(n, kv, Hq, Hkv, D, cancel, seed=81):
    """Keys in pairs 16 apart, which get the same weight; cancel: their values are opposite, so that what is left of
    a row is what its weights are off by; else all values are positive, so that the weights' errors add up."""
    b = Batch(n, kv, kv, Hq, Hkv, D, 64, seed=seed)
    for s, total in enumerate(kv):
        for j in range(total):
            at, lead = (b.table[s, j // 64], j % 64), j - 16 if j // 16 % 2 else j
            of = (b.table[s, lead // 64], lead % 64)
            b.k[at] = b.k[of]
            b.v[at] = b.v[of].abs() * (-1 if cancel and lead != j else 1)
    return b


def definition(b, halves=None):
    """(out, bound): every key seen by every row; halves(weights): what the weights are multiplied as."""
    out = torch.zeros(b.T, b.Hq, b.D, dtype=torch.float64)
    bound = torch.zeros_like(out)
    for s, n in enumerate(b.n):
        keys, vals = (x.double() for x in b.keys(s, b.kv[s]))
        for t in range(int(b.q_start[s]), int(b.q_start[s]) + n):
            for h in range(b.Hq):
                g = h // (b.Hq // b.Hkv)
                x = keys[:, g] @ b.q[t, h].double() * b.scale
                w = torch.exp(x - x.max())
                p = w if halves is None else halves(w.float()).double()
                out[t, h] = p @ vals[:, g] / w.sum()
                bound[t, h] = 2 ** -8 * out[t, h].abs() + WEIGHTS * (w @ vals[:, g].abs()) / w.sum()
    return out, bound


CASES = [([1, 1, 1], [512, 96, 32], 4, 2, 128), ([1], [960], 8, 1, 256), ([1, 4], [640, 256], 4, 1, 128),
         ([20, 3], [512, 128], 4, 2, 128), ([30], [320], 2, 2, 256), ([1], [992], 40, 1, 128)]


def split(w, lost):
    """w as hi + lo, without lo where `lost`."""
    hi = ((w.view(torch.int32) - 0x10000).clamp(min=0) & ~0xFFFF).view(torch.float32)
    lo = (w - hi).bfloat16().float()
    return hi + torch.where(lost, torch.zeros_like(lo), lo)


@pytest.mark.parametrize("D,step", [(128, 128), (256, 64)])
def test_the_bound_notices_a_lost_half(D, step):
    """The bound on the halves as they are, without any low half, and without those of one step of 16 keys a tile."""
    for cancel in (False, True):
        b = batch([2], [512], 2, 1, D, cancel)
        want, bound = definition(b)
        none = torch.zeros(512, dtype=torch.bool)
        got, _ = definition(b, lambda w: split(w, none))
        close(got.bfloat16(), want, bound)
        place = torch.arange(512) % step
        lost = ~none if not cancel else place // 16 == 1
        bad, _ = definition(b, lambda w: split(w, lost))
        with pytest.raises(AssertionError, match="more than the bound"):
            close(bad.bfloat16(), want, bound)


@pytest.mark.gpu
@pytest.mark.parametrize("n,kv,Hq,Hkv,D", CASES)
@pytest.mark.parametrize("cancel", [False, True])
def test_single_kernel(monkeypatch, n, kv, Hq, Hkv, D, cancel):
    from tests.test_gpu_paged import run_attn

    monkeypatch.setenv("DG_PAGED_KERNEL", "single")
    b = batch(n, kv, Hq, Hkv, D, cancel)
    close(run_attn(b, False, 0, False, kv), *definition(b))
