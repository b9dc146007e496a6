"""Inputs of the paged-cache tests and the operators' definitions in 64 bits on the CPU, plain loops over
sequences (no library code)."""
import math

import torch

import block_diffusion_decoding_gb300 as dg

DEV = "cuda"
NAN = float("nan")


class Batch:
    """A ragged batch over a paged cache.  `n` new and `kv` cached tokens of each sequence; `stored` of them have
    their place in the pages.  Every other place of the pages (behind a sequence, other pages) holds NaN, table
    entries past a sequence's last page a page id that does not exist."""

    def __init__(self, n, kv, stored, Hq, Hkv, D, page, seed=0, pad=0, strided=False, extra_width=0):
        g = torch.Generator().manual_seed(seed)
        self.n, self.kv, self.Hq, self.Hkv, self.D, self.page = n, kv, Hq, Hkv, D, page
        B = len(n)
        pages = [-(-s // page) for s in stored]
        self.n_pages = max(1, sum(pages)) + 2
        order = torch.randperm(self.n_pages, generator=g).int()
        self.table = torch.full((B, max(1, max(pages)) + extra_width), -7, dtype=torch.int32)
        at = 0
        for b, m in enumerate(pages):
            self.table[b, :m] = order[at:at + m]
            at += m
        self.k = torch.full((self.n_pages, page, Hkv, D), NAN, dtype=torch.bfloat16)
        self.v = self.k.clone()
        for b in range(B):
            for j0 in range(0, kv[b], page):
                m = min(page, kv[b] - j0)
                self.k[self.table[b, j0 // page], :m] = torch.randn(m, Hkv, D, generator=g).bfloat16()
                self.v[self.table[b, j0 // page], :m] = torch.randn(m, Hkv, D, generator=g).bfloat16()
        self.q_start = torch.tensor([0] + [sum(n[:b + 1]) for b in range(B)], dtype=torch.int32)
        self.T = sum(n) + pad
        self.q = (2 * torch.randn(self.T, Hq, D, generator=g)).bfloat16()
        self.kn = torch.randn(self.T, Hkv, D, generator=g).bfloat16()
        self.vn = torch.randn(self.T, Hkv, D, generator=g).bfloat16()
        for t in (self.q, self.kn, self.vn):   # rows of nobody
            t[sum(n):] = NAN
        self.scale = 1.0 / math.sqrt(D)
        self.strided = strided

    def cache(self, kv=None):
        kv = torch.tensor(self.kv if kv is None else kv, dtype=torch.int32, device=DEV)
        k, v = self.k, self.v
        if self.strided:   # keys and values of a page side by side, two layers' pages interleaved
            both = torch.full((self.n_pages, 2, 2, self.page, self.Hkv, self.D), NAN, dtype=torch.bfloat16,
                              device=DEV)
            both[:, 1, 0], both[:, 1, 1] = k.to(DEV), v.to(DEV)
            return dg.PagedCache(both[:, 1, 0], both[:, 1, 1], self.table.to(DEV), kv, self.q_start.to(DEV))
        return dg.PagedCache(k.to(DEV), v.to(DEV), self.table.to(DEV), kv, self.q_start.to(DEV))

    def rows(self, x, extra=24):
        """x [T, heads, D] on the GPU, as columns of a wider tensor when the batch is strided."""
        if not self.strided:
            return x.to(DEV)
        T, H, D = x.shape
        wide = torch.full((T, H * D + extra), NAN, dtype=torch.bfloat16, device=DEV)
        wide[:, 8:8 + H * D] = x.reshape(T, H * D).to(DEV)
        return wide[:, 8:8 + H * D].view(T, H, D)

    def keys(self, b, stored):
        """The first `stored` keys and values of sequence b."""
        pages = self.table[b, :-(-stored // self.page)].long() if stored else torch.zeros(0, dtype=torch.long)
        return self.k[pages].flatten(0, 1)[:stored], self.v[pages].flatten(0, 1)[:stored]


def attention(batch, causal, window, fresh, stored):
    """(out, bound) [T, Hq, D] in 64 bits: the definition over the visible keys alone, and how far a result in
    bf16 may be off: its own rounding (2^-8 of the value), each weight rounded to bf16 before the product with V
    (2^-8 of sum w |v|), and fp32 scores, exponentials and sums (2^-12 of it: a score of magnitude below 64 held
    in fp32 with D products is within 2^-14 of it in base 2)."""
    out = torch.full((batch.T, batch.Hq, batch.D), NAN, dtype=torch.float64)
    bound = torch.zeros_like(out)
    G = batch.Hq // batch.Hkv
    for b, n in enumerate(batch.n):
        t0 = int(batch.q_start[b])
        keys, vals = batch.keys(b, stored[b])
        if fresh:
            keys = torch.cat([keys, batch.kn[t0:t0 + n]])
            vals = torch.cat([vals, batch.vn[t0:t0 + n]])
        N = keys.shape[0]
        for h in range(batch.Hq):
            K, V = keys[:, h // G].double(), vals[:, h // G].double()
            for i in range(n):
                pos = N - n + i
                hi = min(N, pos + 1) if causal else N
                lo = max(0, pos - window + 1) if window else 0
                if hi <= lo:
                    out[t0 + i, h] = 0
                    continue
                s = K[lo:hi] @ batch.q[t0 + i, h].double() * batch.scale
                w = torch.softmax(s, 0)
                out[t0 + i, h] = w @ V[lo:hi]
                bound[t0 + i, h] = 2 ** -8 * out[t0 + i, h].abs() + (2 ** -8 + 2 ** -12) * (w @ V[lo:hi].abs())
    return out, bound


def norm_rope(x, positions, inv_freq, interleaved, weight, eps, offset):
    """(y, bound) of heads x [T, H, D] in 64 bits; bound: the rounding to bf16 (2^-8) and fp32 arithmetic with
    sines and cosines within 2^-20 (2^-17 of the pair's length covers the norm, the products and the angle)."""
    x = x.double()
    if weight is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * (offset + weight.double())
    y, size = x.clone(), x.abs().clone()
    half = 0 if inv_freq is None else len(inv_freq)
    for m in range(half):
        a, b = (2 * m, 2 * m + 1) if interleaved else (m, m + half)
        phi = (positions.double() * inv_freq[m])[:, None]
        y[..., a] = x[..., a] * phi.cos() - x[..., b] * phi.sin()
        y[..., b] = x[..., b] * phi.cos() + x[..., a] * phi.sin()
        size[..., a] = size[..., b] = torch.hypot(x[..., a], x[..., b])
    return y, 2 ** -8 * y.abs() + 2 ** -17 * size


def inv_freq(rot, theta=10000.0):
    return theta ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot) if rot else None


def close(got, want, bound):
    got = got.double().cpu()
    off = (got - want).abs() - bound
    assert torch.isfinite(got).all(), "not finite"
    assert (off <= 0).all(), "off by %.3g more than the bound at %s" % (
        off.max(), tuple(torch.nonzero(off == off.max())[0].tolist()))
