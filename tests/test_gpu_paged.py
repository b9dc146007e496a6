"""GPU tests of the paged-cache operators against their definitions in 64 bits: dg_qk_norm_rope,
dg_paged_append and dg_paged_attn, alone and as a server of block diffusion chains them."""
import pytest
import torch

import block_diffusion_decoding_gb300 as dg
from tests._helpers import status_ok
from tests._paged import DEV, NAN, Batch, attention, close, inv_freq, norm_rope

pytestmark = pytest.mark.gpu


def same_bits(a, b):
    return torch.equal(a.contiguous().view(torch.int16).cpu(), b.contiguous().view(torch.int16).cpu())


# ---------------------------------------------------------------- norm and rotation
def heads_of(T, H, D, seed):
    g = torch.Generator().manual_seed(seed)
    return (3 * torch.randn(T, H, D, generator=g)).bfloat16()


@pytest.mark.parametrize("T,Hq,Hkv,D,rot,interleaved,normed,offset", [
    (1, 4, 1, 128, 128, False, True, 1.0),
    (1, 1, 1, 16, 16, True, True, 0.0),
    (7, 3, 2, 80, 32, False, True, 1.0),
    (33, 5, 1, 256, 64, True, False, 0.0),
    (257, 16, 8, 256, 256, False, True, 1.0),
    (5, 16, 8, 128, 0, False, True, 0.0),
    (3, 2, 1, 48, 16, False, True, 0.0),
    (9001, 9, 3, 128, 96, False, True, 0.0),     # several heads a lane group, not a multiple of them
    (3500, 17, 8, 256, 256, False, True, 1.0),   # twice as many
    (7001, 17, 8, 128, 64, True, True, 1.0),
])
@pytest.mark.parametrize("strided", [False, True])
def test_norm_rope(T, Hq, Hkv, D, rot, interleaved, normed, offset, strided):
    b = Batch([T], [0], [0], Hq, Hkv, D, 16, strided=strided)
    q, k = heads_of(T, Hq, D, 1), heads_of(T, Hkv, D, 2)
    g = torch.Generator().manual_seed(3)
    pos = torch.randint(0, 262144, (T,), generator=g, dtype=torch.int32)
    pos[0] = 262143
    qw, kw = ((0.5 * torch.randn(D, generator=g)).bfloat16() for _ in range(2)) if normed else (None, None)
    f = inv_freq(rot)
    p = dg.head_params(Hq, Hkv, D, rope_steps=None if f is None else dg.rope_steps(f, DEV), interleaved=interleaved,
                       q_weight=qw.to(DEV) if normed else None, k_weight=kw.to(DEV) if normed else None, eps=1e-5,
                       weight_offset=offset)
    qd, kd = b.rows(q), b.rows(k)
    qo, ko = b.rows(torch.full_like(q, NAN)), b.rows(torch.full_like(k, NAN))
    dg.qk_norm_rope(qd, kd, qo, ko, pos.to(DEV), p)
    close(qo, *norm_rope(q, pos, f, interleaved, qw, 1e-5, offset))
    close(ko, *norm_rope(k, pos, f, interleaved, kw, 1e-5, offset))
    assert same_bits(qd, q) and same_bits(kd, k)
    # in place, and one of the two alone
    only = b.rows(torch.full_like(k, NAN))
    dg.qk_norm_rope(None, kd, None, only, pos.to(DEV), p)
    assert same_bits(only, ko)
    dg.qk_norm_rope(qd, kd, qd, kd, pos.to(DEV), p)
    assert same_bits(qd, qo) and same_bits(kd, ko)


def test_norm_rope_extremes():
    """Zero heads stay zero; negative and the largest positions; a head whose squares stay below the smallest
    normal number keeps eps in charge; heads with infinities and NaN leave the other heads alone."""
    D, f = 128, inv_freq(128)
    x = torch.zeros(6, 2, D)
    g = torch.Generator().manual_seed(5)
    x[1:] = torch.randn(5, 2, D, generator=g)
    x[3] *= 1e-25
    x = x.bfloat16()
    pos = torch.tensor([5, -1, 2 ** 31 - 1, 7, -2 ** 31, 0], dtype=torch.int32)
    w = torch.ones(D, dtype=torch.bfloat16)
    p = dg.head_params(2, 1, D, rope_steps=dg.rope_steps(f, DEV), q_weight=w.to(DEV), eps=1e-6)
    out = torch.full_like(x, NAN).to(DEV)
    dg.qk_norm_rope(x.to(DEV), None, out, None, pos.to(DEV), p)
    # at |position| 2^31 the 64-bit reference's own angle is off by 2^31 2^-53 times a few: far below the bound
    close(out, *norm_rope(x, pos, f, False, w, 1e-6, 0.0))
    y = x.clone()
    y[1, 0, 3], y[2, 1, 100] = float("inf"), NAN
    bad = torch.full_like(x, NAN).to(DEV)
    dg.qk_norm_rope(y.to(DEV), None, bad, None, pos.to(DEV), p)
    keep = torch.ones(6, 2, dtype=torch.bool)
    keep[1, 0] = keep[2, 1] = False
    assert same_bits(bad.cpu()[keep], out.cpu()[keep])
    # no tokens
    e = torch.empty(0, 2, D, dtype=torch.bfloat16, device=DEV)
    dg.qk_norm_rope(e, None, e, None, torch.empty(0, dtype=torch.int32, device=DEV), p)


@pytest.mark.parametrize("interleaved", [False, True])
def test_infinities_outside_the_rotation_stay(interleaved):
    """A value that is not rotated meets no product with its neighbour: an infinity there stays one value."""
    D, rot = 128, 64
    x = heads_of(4, 2, D, 6)
    x[1, 0, 65], x[2, 1, 127] = float("inf"), float("-inf")
    pos = torch.arange(4, dtype=torch.int32)
    p = dg.head_params(2, 1, D, rope_steps=dg.rope_steps(inv_freq(rot), DEV), interleaved=interleaved)
    out = torch.full_like(x, NAN).to(DEV)
    dg.qk_norm_rope(x.to(DEV), None, out, None, pos.to(DEV), p)
    assert torch.equal(out.cpu()[..., rot:], x[..., rot:])


# ---------------------------------------------------------------- append
@pytest.mark.parametrize("n,kv,Hq,Hkv,D,page,rot,interleaved,pad", [
    ([1], [0], 4, 1, 128, 16, 128, False, 0),
    ([1, 1, 1, 1], [15, 16, 300, 31], 4, 2, 128, 16, 64, True, 3),
    ([5, 0, 40, 17], [0, 20, 47, 90], 16, 8, 256, 48, 256, False, 2),
    ([300, 1], [700, 63], 3, 1, 256, 64, 32, True, 0),
    ([400, 1, 700], [10, 0, 77], 6, 2, 256, 32, 128, False, 0),
    ([2500, 1, 900, 4000], [13, 2047, 5, 0], 16, 8, 128, 128, 128, False, 1),
    ([1700, 1200], [100, 0], 11, 9, 256, 64, 64, True, 2),
])
@pytest.mark.parametrize("strided", [False, True])
def test_append(n, kv, Hq, Hkv, D, page, rot, interleaved, pad, strided):
    total = [a + b for a, b in zip(n, kv)]
    b = Batch(n, kv, total, Hq, Hkv, D, page, seed=9, pad=pad, strided=strided, extra_width=1)
    f = inv_freq(rot)
    g = torch.Generator().manual_seed(4)
    qw, kw = ((1 + 0.2 * torch.randn(D, generator=g)).bfloat16() for _ in range(2))
    p = dg.head_params(Hq, Hkv, D, rope_steps=dg.rope_steps(f, DEV), interleaved=interleaved, q_weight=qw.to(DEV),
                       k_weight=kw.to(DEV), eps=1e-6)
    c = b.cache()
    k0, v0 = c.k.cpu(), c.v.cpu()
    ws = dg.workspace(dg.paged_append_workspace(), DEV)
    qo = b.rows(torch.full_like(b.q, 7.0))
    lens = torch.zeros(len(n), dtype=torch.int32, device=DEV)
    dg.paged_append(b.rows(b.kn), b.rows(b.vn), c, p, ws, q=b.rows(b.q), q_out=qo, kv_len_out=lens)
    status_ok(ws)
    assert lens.tolist() == total
    place = torch.cat([torch.arange(kv[i], total[i]) for i in range(len(n))])
    seq = torch.cat([torch.full((m,), i) for i, m in enumerate(n)])
    T = sum(n)
    pages, at = b.table[seq, place // page].long(), place % page
    want, bound = norm_rope(b.kn[:T], place, f, interleaved, kw, 1e-6, 0.0)
    close(c.k.cpu()[pages, at], want, bound)
    assert same_bits(c.v.cpu()[pages, at], b.vn[:T])
    close(qo[:T], *norm_rope(b.q[:T], place, f, interleaved, qw, 1e-6, 0.0))
    assert (qo[T:] == 7.0).all()                 # rows of nobody: as they were
    # every other place of the pages is untouched
    kept = torch.ones(b.n_pages, page, dtype=torch.bool)
    kept[pages, at] = False
    assert same_bits(c.k.cpu()[kept], k0[kept]) and same_bits(c.v.cpu()[kept], v0[kept])
    # positions of its own; keys and values alone
    pos = torch.arange(b.T, dtype=torch.int32) * 3 + 1000
    c2 = b.cache()
    dg.paged_append(b.rows(b.kn), b.rows(b.vn), c2, p, ws, positions=pos.to(DEV))
    close(c2.k.cpu()[pages, at], *norm_rope(b.kn[:T], pos[:T], f, interleaved, kw, 1e-6, 0.0))
    status_ok(ws)


def test_append_copies_bits_without_norm_and_rotation():
    b = Batch([6, 3], [1, 20], [7, 23], 2, 2, 128, 16, seed=2)
    b.kn.view(torch.int16)[0, 0, :4] = torch.tensor([0x7F81, -1, 0x7F80, 1], dtype=torch.int16)   # NaN payloads
    b.vn.view(torch.int16)[0, 0, :4] = torch.tensor([0x7F81, -1, 0x7F80, 1], dtype=torch.int16)
    c = b.cache()
    ws = dg.workspace(256, DEV)
    dg.paged_append(b.kn.to(DEV), b.vn.to(DEV), c, dg.head_params(2, 2, 128), ws)
    b.k, b.v = c.k.cpu(), c.v.cpu()
    for i, (n, kv) in enumerate(zip(b.n, b.kv)):
        t = int(b.q_start[i])
        k, v = b.keys(i, kv + n)
        assert same_bits(k[kv:], b.kn[t:t + n]) and same_bits(v[kv:], b.vn[t:t + n])


def test_append_reports_places_it_cannot_store():
    """A page id outside the cache, a place past the table and lengths that do not fit: reported, and nothing
    else is written (the kernel checks each before it stores)."""
    b = Batch([4, 4], [14, 0], [18, 4], 2, 1, 128, 16, seed=3)
    ws = dg.workspace(256, DEV)
    p = dg.head_params(2, 1, 128)
    for table, kv, start in (([[0, 99], [1, 0]], [14, 0], [0, 4, 8]), ([[0, -1], [1, 0]], [14, 0], [0, 4, 8]),
                             ([[0, 2], [1, 0]], [30, 0], [0, 4, 8]), ([[0, 2], [1, 0]], [-6, 0], [0, 4, 8]),
                             ([[0, 2], [1, 0]], [14, 0], [0, 4, 90])):
        c = b.cache(kv)
        c.page_table.copy_(torch.tensor(table, dtype=torch.int32))
        c.q_start.copy_(torch.tensor(start, dtype=torch.int32))
        k0 = c.k.clone()
        dg.paged_append(b.kn.to(DEV), b.vn.to(DEV), c, p, ws)
        assert dg.read_device_status(ws, clear=True) == 7
        k, want = c.k.cpu(), k0.cpu()
        for s in range(2):
            for i in range(4):
                at = kv[s] + i
                if 0 <= at < 32 and 0 <= table[s][at // 16] < b.n_pages:
                    want[table[s][at // 16], at % 16] = b.kn[4 * s + i]
        assert same_bits(k, want)


# ---------------------------------------------------------------- attention
def run_attn(b, causal, window, fresh, stored, out=None, ws=None):
    c = b.cache(stored)
    ws = dg.workspace(dg.paged_attn_workspace(b.T, b.Hq, c), DEV) if ws is None else ws
    out = b.rows(torch.full_like(b.q, 5.0)) if out is None else out
    dg.paged_attn(b.rows(b.q), c, out, b.scale, ws, k_new=b.rows(b.kn) if fresh else None,
                  v_new=b.rows(b.vn) if fresh else None, causal=causal, window=window)
    torch.cuda.synchronize()
    status_ok(ws)
    return out


def check_attn(n, kv, Hq, Hkv, D, page, causal, window, fresh, pad=0, strided=False, seed=0):
    """kv: cached tokens; with fresh the new tokens' keys come beside them, else they are the last n of kv."""
    b = Batch(n, kv, kv, Hq, Hkv, D, page, seed=seed, pad=pad, strided=strided, extra_width=pad)
    out = run_attn(b, causal, window, fresh, kv)
    T = sum(n)
    want, bound = attention(b, causal, window, fresh, kv)
    close(out[:T], want[:T], bound[:T])
    assert (out[T:] == 5.0).all()                # rows of nobody: as they were
    return b, out


@pytest.fixture(params=["single", "pair"])
def kernel(request, monkeypatch):
    """Query tiles of 128 rows on one CTA, or of 256 on two."""
    monkeypatch.setenv("DG_PAGED_KERNEL", request.param)


MASKS = [(False, 0, False), (False, 0, True), (True, 0, False), (True, 0, True), (True, 5, False), (True, 130, True)]


@pytest.mark.parametrize("causal,window,fresh", MASKS)
@pytest.mark.parametrize("Hq,Hkv,D", [(2, 1, 128), (6, 2, 256), (5, 1, 128), (4, 4, 256)])
def test_attention_small_and_ragged(kernel, Hq, Hkv, D, causal, window, fresh):
    """Lengths around tiles, pages and nothing: empty sequences, empty caches, one token, tails of a tile."""
    n = [1, 0, 7, 33, 1, 2, 1]
    kv = [1, 9, 0, 40, 129, 64, 0]
    if not fresh:
        kv = [k + m for k, m in zip(kv, n)]
    check_attn(n, kv, Hq, Hkv, D, 16, causal, window, fresh, pad=3, seed=1)
    check_attn(n, kv, Hq, Hkv, D, 48, causal, window, fresh, strided=True, seed=2)


@pytest.mark.parametrize("causal,window,fresh", MASKS)
@pytest.mark.parametrize("page", [16, 64, 256])
@pytest.mark.parametrize("D", [128, 256])
def test_attention_cut_between_ctas(kernel, D, page, causal, window, fresh):
    """Long caches and several query tiles: items cut between CTAs and merged."""
    n, kv = [70, 1, 130], [900, 2500, 333]
    if not fresh:
        kv = [k + m for k, m in zip(kv, n)]
    check_attn(n, kv, 4, 2, D, page, causal, window, fresh, seed=3)


@pytest.mark.parametrize("n,kv,Hq,Hkv,D,causal,window,fresh",
                         [([640, 600], [1200, 500], 32, 8, 128, *m) for m in MASKS[:4] + [(True, 300, False)]]
                         + [([0, 1500, 1], [40, 500, 7], 24, 8, 256, True, 0, True)])
def test_attention_whole_items_then_a_cut_rest(n, kv, Hq, Hkv, D, causal, window, fresh):
    """More than two query tiles for every CTA pair, of unequal cost: whole ones in turn, then the cut rest."""
    tiles = sum(-(-m * (Hq // Hkv) // 256) * Hkv for m in n)
    units = torch.cuda.get_device_properties(0).multi_processor_count // 2
    assert tiles >= max(16 * len(n), 2 * units)
    if not fresh:
        kv = [k + m for k, m in zip(kv, n)]
    check_attn(n, kv, Hq, Hkv, D, 64, causal, window, fresh, seed=9)


@pytest.mark.parametrize("D,Hq,Hkv", [(128, 4, 1), (256, 16, 8), (128, 128, 1), (256, 40, 2)])
def test_attention_single_tokens(D, Hq, Hkv):
    check_attn([1] * 9, [1, 2, 17, 128, 700, 1500, 64, 31, 4100], Hq, Hkv, D, 32, True, 0, False, seed=4)


@pytest.mark.parametrize("D,Hkv", [(128, 1), (256, 2)])
def test_attention_one_long_sequence(D, Hkv):
    """One token over a cache that every CTA takes a stretch of."""
    check_attn([1], [20000], 2 * Hkv, Hkv, D, 64, True, 0, False, seed=5)


@pytest.mark.parametrize("wide", [False, True])
def test_whole_items_of_many_sequences(wide, monkeypatch):
    """More than 32 sequences with 16 items each and more, on CTA pairs; wide: a table of so many pages that the
    work is divided in 64 bits."""
    monkeypatch.setenv("DG_PAGED_KERNEL", "pair")
    g = torch.Generator().manual_seed(31)
    n = torch.randint(10, 40, (33,), generator=g).tolist()[:-2] + [140, 150]
    kv = [m + int(k) for m, k in zip(n, torch.randint(10, 200, (33,), generator=g))]
    check_attn_wide(n, kv, 32, 16, 128, 2048 if wide else 16, 1 << 14 if wide else 0)


@pytest.mark.parametrize("n,kv,Hq,Hkv,D", [([1, 3, 1], [900, 64, 1], 16, 8, 128), ([90, 1, 200], [900, 64, 700], 6, 2, 256)])
def test_division_in_64_bits(kernel, n, kv, Hq, Hkv, D):
    """The same work with a table of 2^25 tokens' pages and with one that just fits: the same bits."""
    kv = [max(k, m) for k, m in zip(kv, n)]
    assert same_bits(check_attn_wide(n, kv, Hq, Hkv, D, 64, 1 << 19), check_attn_wide(n, kv, Hq, Hkv, D, 64, 0))


def check_attn_wide(n, kv, Hq, Hkv, D, page, extra):
    b = Batch(n, kv, kv, Hq, Hkv, D, page, seed=32, extra_width=extra)
    out = run_attn(b, True, 0, False, kv)
    want, bound = attention(b, True, 0, False, kv)
    close(out, want, bound)
    return out.cpu()


def test_rows_that_see_nothing_are_zero(kernel):
    """Causal, with more new tokens than cached keys (their keys were not all appended): the first rows see none."""
    b, out = check_attn([12, 3], [5, 0], 4, 2, 128, 16, True, 0, False, seed=6)
    assert (out[:7] == 0).all() and (out[12:] == 0).all()


def test_many_sequences(kernel):
    g = torch.Generator().manual_seed(8)
    n = torch.randint(0, 4, (531,), generator=g).tolist()
    kv = [int(x) + m for x, m in zip(torch.randint(0, 90, (531,), generator=g), n)]
    check_attn(n, kv, 2, 1, 128, 16, True, 0, False, seed=8)


@pytest.mark.parametrize("D,Hq,Hkv,page", [(128, 2, 1, 16), (256, 6, 2, 64), (128, 1, 1, 48), (256, 4, 4, 128)])
@pytest.mark.parametrize("window,fresh", [(0, False), (0, True), (130, True), (70, False)])
def test_values_that_are_not_finite_stay_with_the_rows_that_see_them(kernel, D, Hq, Hkv, page, window, fresh):
    """Infinities and NaN in the keys and values of some tokens: the rows that do not see such a token are as if it
    were not there; the others get what the definition gives (an infinite value: that infinity; a NaN: NaN)."""
    n, kv = [150, 1, 90, 300], [700, 300, 0, 33]
    if not fresh:
        kv = [k + m for k, m in zip(kv, n)]
    b = Batch(n, kv, kv, Hq, Hkv, D, page, seed=50, strided=True)

    def put(s, key, dim, value, which):
        """A value into key `key` (of all the sequence's keys) of sequence s."""
        if key < kv[s]:
            pages = b.k if which == "k" else b.v
            pages[b.table[s, key // page], key % page, 0, dim] = value
        else:
            (b.kn if which == "k" else b.vn)[int(b.q_start[s]) + key - kv[s], 0, dim] = value

    total = [k + (m if fresh else 0) for k, m in zip(kv, n)]
    inf = float("inf")
    put(0, total[0] - 20, 3, inf, "v")              # a late token: hidden from the rows before it
    put(0, total[0] - 60, D - 1, -inf, "v")
    put(0, total[0] - 100, 1, NAN, "k")             # a key: its score is NaN where it is seen
    put(0, total[0] - 200, D // 2, NAN, "v")        # behind the window of the later rows, where there is one
    put(2, 40, 0, NAN, "v")
    put(3, total[3] - 1, D // 2 + 1, inf, "v")      # the last token: only its own row sees it
    put(3, total[3] - 299, 5, -inf, "v")
    out = run_attn(b, True, window, fresh, kv).cpu().double()
    want, bound = attention(b, True, window, fresh, kv)
    assert torch.equal(torch.isnan(out), torch.isnan(want))
    ends = torch.isinf(want)
    assert torch.equal(out[ends], want[ends]) and ends.any() and torch.isnan(want).any()
    fine = torch.isfinite(want)
    off = (out[fine] - want[fine]).abs() - bound[fine]
    assert torch.isfinite(out[fine]).all() and (off <= 0).all(), off.max()


@pytest.mark.parametrize("D,Hq,Hkv,page", [(128, 2, 1, 16), (256, 8, 1, 64), (128, 16, 1, 48), (256, 4, 4, 128)])
@pytest.mark.parametrize("window,causal", [(0, True), (0, False), (200, True)])
def test_infinite_values_that_single_tokens_see(kernel, D, Hq, Hkv, page, window, causal):
    """Infinities and NaN among the values in every part of a tile: the dims that have them get what the
    definition gives, the other dims and the other sequences their sums."""
    kv = [513, 128, 300, 77, 64]
    b = Batch([1] * 5, kv, kv, Hq, Hkv, D, page, seed=57, strided=True)
    at = {}

    def put(s, key, dim, value):
        assert b.v[b.table[s, key // page], key % page, 0, dim].isfinite() and (s, dim) not in at
        b.v[b.table[s, key // page], key % page, 0, dim] = value
        at[s, dim] = value

    inf = float("inf")
    for j, key in enumerate((512, 500, 470, 440, 410)):       # each quarter of a tile, and its last, short one
        put(0, key, 7 + 17 * j, inf if j & 1 else -inf)
    put(0, 400, 127, NAN)
    put(0, 3, 126, inf)                                       # behind the window, where there is one
    put(2, 299, 0, -inf)
    put(3, 0, D - 1, inf)
    put(3, 76, D - 2, NAN)
    out = run_attn(b, causal, window, False, kv).cpu().double()
    want, bound = attention(b, causal, window, False, kv)
    assert torch.equal(torch.isnan(out), torch.isnan(want)) and torch.isnan(want).any()
    ends = torch.isinf(want)
    assert torch.equal(out[ends], want[ends]) and ends.any()
    fine = torch.isfinite(want)
    assert torch.isfinite(out[fine]).all() and ((out[fine] - want[fine]).abs() <= bound[fine]).all()


def test_scores_far_apart(kernel):
    """Scores from -1000 to 1000 in an order that moves the reference maximum late, and large negative ones only."""
    b = Batch([40], [600], [600], 2, 1, 128, 64, seed=10)
    ramp = torch.linspace(-1, 1, 640)
    k, _ = b.keys(0, 600)
    b.q[:] = 0
    b.q[:, :, 0] = 100
    for sign in (1, -1):
        for j in range(600):
            b.k[b.table[0, j // 64], j % 64, 0, 0] = (sign * 100 * ramp[j] - (120 if sign < 0 else 0)).bfloat16()
        b.kn[:40, 0, 0] = (sign * 100 * ramp[600:] - (120 if sign < 0 else 0)).bfloat16()
        out = run_attn(b, False, 0, True, [600])
        want, _ = attention(b, False, 0, True, [600])
        # a score s (base 2) of magnitude up to 2^13 is within 2^-10 in fp32: weights within 2^-10 ln 2 < 2^-10
        vmax = max(b.keys(0, 600)[1].double().abs().max(), b.vn[:40].double().abs().max())
        close(out, want, (2 ** -8 + 2 ** -8 + 2 ** -9) * vmax * torch.ones_like(want))


def test_results_do_not_depend_on_pages_or_repeats():
    """Page order, page size and a second run change no bit (where the division of the work is the same)."""
    n, kv = [64, 1, 200], [777, 3000, 100]
    outs = []
    for page, seed in ((16, 1), (64, 1), (128, 1)):
        b = Batch(n, kv, kv, 4, 2, 128, page, seed=seed)
        g = torch.Generator().manual_seed(77)
        for s in range(3):          # the same keys in every layout
            for j in range(kv[s]):
                b.k[b.table[s, j // page], j % page] = torch.randn(2, 128, generator=g).bfloat16()
                b.v[b.table[s, j // page], j % page] = torch.randn(2, 128, generator=g).bfloat16()
        b.q = torch.randn(b.T, 4, 128, generator=torch.Generator().manual_seed(5)).bfloat16()
        for _ in range(2):
            outs.append(run_attn(b, True, 0, False, kv))
    for o in outs[1:]:
        assert same_bits(o, outs[0])


def test_attention_reports_bad_pages_and_lengths(kernel):
    b = Batch([2, 2], [40, 20], [40, 20], 2, 1, 128, 16, seed=12)
    c = b.cache()
    ws = dg.workspace(dg.paged_attn_workspace(b.T, 2, c), DEV)
    out = torch.zeros_like(b.q, device=DEV)

    def status(table=None, kv=None, start=None):
        d = b.cache(kv)
        if table is not None:
            d.page_table[0, 1] = table
        if start is not None:
            d.q_start.copy_(torch.tensor(start, dtype=torch.int32))
        dg.paged_attn(b.q.to(DEV), d, out, b.scale, ws)
        return dg.read_device_status(ws, clear=True)

    assert status() == 0
    good = out.clone()
    assert status(table=b.n_pages) == 7 and status(table=-1) == 7
    assert status(kv=[40, 10 ** 9]) == 7 and status(kv=[-1, 20]) == 7
    assert status(start=[0, 2, 100]) == 7 and status(start=[-4, 2, 4]) == 7
    out.fill_(0)
    assert status() == 0 and same_bits(out, good)


@pytest.mark.parametrize("D", [128, 256])
def test_rows_that_decrease_compute_nothing(kernel, D):
    """q_start must not decrease: the sequences' rows could add up to more than the division of the work was
    measured for.  Reported, and the output is left as it was; the workspace then serves a good batch."""
    B = 40
    b = Batch([3] * B, [50] * B, [50] * B, 4, 2, D, 16, seed=13)
    c, d = b.cache(), b.cache()
    d.q_start.copy_(torch.tensor([(0, b.T)[i & 1] for i in range(B + 1)], dtype=torch.int32))
    ws = dg.workspace(dg.paged_attn_workspace(b.T, 4, c), DEV)
    out = torch.full_like(b.q, 5.0).to(DEV)
    dg.paged_attn(b.q.to(DEV), d, out, b.scale, ws)
    assert dg.read_device_status(ws, clear=True) == 7 and (out == 5).all()
    dg.paged_attn(b.q.to(DEV), c, out, b.scale, ws)
    status_ok(ws)
    want, bound = attention(b, True, 0, False, b.kv)
    close(out, want, bound)


def test_rows_before_the_first_sequence_are_left(kernel):
    """q_start[0] > 0: a batch whose first rows belong to nobody."""
    b = Batch([4, 1, 9], [80, 33, 200], [80, 33, 200], 4, 2, 128, 16, seed=21)
    want, bound = attention(b, True, 0, False, b.kv)
    lead = torch.full((5, 4, 128), float("nan"), dtype=torch.bfloat16)
    c = b.cache()
    c.q_start += 5
    q = torch.cat([lead, b.q]).to(DEV)
    out = torch.full_like(q, 5.0)
    ws = dg.workspace(dg.paged_attn_workspace(len(q), 4, c), DEV)
    dg.paged_attn(q, c, out, b.scale, ws)
    status_ok(ws)
    close(out[5:], want, bound)
    assert (out[:5] == 5).all()
    # the append's rows likewise: the same tokens as from row 0 on
    k, v = (torch.cat([lead[:, :2], t]).to(DEV) for t in (b.kn, b.vn))
    d, p, wa = b.cache([76, 32, 191]), dg.head_params(4, 2, 128), dg.workspace(256, DEV)
    e = b.cache([76, 32, 191])
    dg.paged_append(b.kn.to(DEV), b.vn.to(DEV), e, p, wa)
    d.q_start += 5
    qo = torch.full_like(q, 5.0)
    dg.paged_append(k, v, d, p, wa, q=q, q_out=qo)
    status_ok(wa)
    assert same_bits(d.k.cpu(), e.k.cpu()) and same_bits(d.v.cpu(), e.v.cpu())
    assert same_bits(qo[5:].cpu(), b.q) and (qo[:5] == 5).all()


@pytest.mark.parametrize("page", [2048, 2032])
def test_the_largest_pages(kernel, page):
    for D, causal, window, fresh in ((128, True, 0, False), (256, False, 0, True), (256, True, 900, False)):
        check_attn([1, 140, 3], [2500, 4100, 2047], 4, 2, D, page, causal, window, fresh, seed=22)


def test_expanded_tensors_are_refused():
    b = Batch([1, 1], [20, 20], [20, 20], 2, 1, 128, 16, seed=23)
    c, ws = b.cache(), dg.workspace(1 << 22, DEV)
    q, out = b.q.to(DEV), torch.empty_like(b.q, device=DEV)
    with pytest.raises(dg.DgError):
        dg.paged_attn(q[:1].expand(2, 2, 128), c, out, b.scale, ws)
    with pytest.raises(dg.DgError):
        dg.paged_attn(q, c, out, b.scale, ws.cpu())
    with pytest.raises(dg.DgError):
        dg.qk_norm_rope(q, None, out, None, torch.zeros(2, dtype=torch.int32, device=DEV),
                        dg.head_params(2, 1, 128, rope_steps=dg.rope_steps([1.0] * 8, "cpu")))
    with pytest.raises(dg.DgError):
        dg.PagedCache(c.k[:1].expand_as(c.k), c.v[:1].expand_as(c.v), c.page_table, c.kv_len, c.q_start)


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("n,kv", [([1, 1, 1], [300, 5000, 64]), ([40, 200, 1], [300, 5000, 64])])
def test_device_checks(kernel, D, n, kv):
    """With dg_set_device_checks on, finite inputs report nothing and give the same bits; an infinite query is
    reported (and goes unreported with the checks off)."""
    b = Batch(n, kv, kv, 4, 2, D, 64, seed=24)
    plain = run_attn(b, True, 0, False, kv)
    c, out = b.cache(), torch.empty_like(b.q, device=DEV)
    ws = dg.workspace(dg.paged_attn_workspace(b.T, 4, c), DEV)
    q = b.q.to(DEV)
    odd = q.clone()
    odd[n[0], 1, 3] = float("inf")
    for x, on, status in ((q, True, 0), (odd, True, 7), (odd, False, 0)):
        dg.set_device_checks(on)
        try:
            dg.paged_attn(x, c, out, b.scale, ws)
        finally:
            dg.set_device_checks(False)
        assert dg.read_device_status(ws, clear=True) == status
        if x is q:
            assert same_bits(out.cpu(), plain.cpu())


# ---------------------------------------------------------------- streams, graphs, the chain
def test_captured_graph_follows_lengths_and_table():
    """One captured append + attention, replayed as the sequences grow, on another stream's capture; two graphs
    over one workspace, replayed in turn, and an eager call between them."""
    Hq, Hkv, D, page = 4, 2, 128, 16
    n, kv = [1, 1, 1], [15, 40, 0]
    final = [k + 3 for k in kv]
    b = Batch(n, kv, final, Hq, Hkv, D, page, seed=14)
    c = b.cache(kv)
    after = torch.zeros(3, dtype=torch.int32, device=DEV)
    read = dg.PagedCache(c.k, c.v, c.page_table, after, c.q_start)
    p = dg.head_params(Hq, Hkv, D, rope_steps=dg.rope_steps(inv_freq(64), DEV))
    ws = dg.workspace(dg.paged_attn_workspace(3, Hq, c), DEV)
    q, kn, vn = b.q.to(DEV), b.kn.to(DEV), b.vn.to(DEV)
    qo, outs = torch.empty_like(q), [torch.empty_like(q) for _ in range(2)]

    def step(out):
        dg.paged_append(kn, vn, c, p, ws, q=q, q_out=qo, kv_len_out=after)
        dg.paged_attn(qo, read, out, b.scale, ws)

    step(outs[0])       # warm: attributes are set outside any capture
    c.kv_len.copy_(torch.tensor(kv, dtype=torch.int32))
    c.k.copy_(b.k)
    c.v.copy_(b.v)
    graphs = []
    side = torch.cuda.Stream()
    for out in outs:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.stream(side):
            torch.cuda.synchronize()
            graph.capture_begin()
            step(out)
            graph.capture_end()
        graphs.append(graph)
    torch.cuda.synchronize()
    eager = torch.empty_like(q)
    for t in range(3):
        g = torch.Generator().manual_seed(100 + t)
        for x in (q, kn, vn):
            x.copy_(torch.randn(*x.shape, generator=g).bfloat16())
        if t == 1:
            step(eager)
        graphs[t % 2].replay()
        torch.cuda.synchronize()
        status_ok(ws)
        b.k, b.v, b.q = c.k.cpu(), c.v.cpu(), qo.cpu()
        now = after.tolist()
        assert now == [k + t + 1 for k in kv]
        want, bound = attention(b, True, 0, False, now)
        close(outs[t % 2], want, bound)
        if t == 1:
            assert same_bits(eager, outs[1])
        c.kv_len.copy_(after)


def test_two_streams_with_their_own_workspaces():
    bs = [Batch([64, 1], [2000 + 50 * i, 900], [2000 + 50 * i, 900], 4, 1, 128, 64, seed=20 + i) for i in range(2)]
    runs = []
    for b in bs:
        c = b.cache()
        runs.append((b, c, dg.workspace(dg.paged_attn_workspace(b.T, 4, c), DEV), b.q.to(DEV),
                     torch.empty_like(b.q, device=DEV), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(5):
        for b, c, ws, q, out, st in runs:
            dg.paged_attn(q, c, out, b.scale, ws, stream=st)
    torch.cuda.synchronize()
    for b, c, ws, q, out, st in runs:
        status_ok(ws)
        want, bound = attention(b, True, 0, False, b.kv)
        close(out, want, bound)


def test_matches_the_dense_cache_operators():
    """A batch of equal lengths: the paged calls agree with dg_canvas_attn and dg_encoder_append on a dense copy of
    the cache, each within its own bound of the definition."""
    B, L, P, Hq, Hkv, D, page = 2, 64, 160, 4, 2, 128, 32
    b = Batch([L] * B, [P] * B, [P] * B, Hq, Hkv, D, page, seed=30)
    want, bound = attention(b, False, 0, True, b.kv)
    close(run_attn(b, False, 0, True, b.kv), want, bound)
    kp = torch.stack([b.keys(i, P)[0] for i in range(B)]).to(DEV)
    vp = torch.stack([b.keys(i, P)[1] for i in range(B)]).to(DEV)
    q, kn, vn = (x.view(B, L, -1, D).to(DEV) for x in (b.q, b.kn, b.vn))
    out = torch.empty_like(q)
    dg.canvas_attn(q, kp, vp, kn, vn, out, b.scale, dg.workspace(dg.canvas_attn_workspace(B, L, P, Hq, Hkv, D), DEV))
    # the dense kernel may also round a key split's partial rows to bf16 once
    close(out.view(B * L, Hq, D), want, 2 * bound)


def test_block_diffusion_over_pages():
    """As a server runs it: canvases of two sequences attend to their pages without a mask (norm and rotation, then
    the attention with the canvas's own keys), are committed (append with norm and rotation), and read back
    causally; three blocks, one sequence starting from nothing."""
    Hq, Hkv, D, page, L, blocks = 4, 2, 128, 32, 40, 3
    kv = [70, 0]
    final = [k + blocks * L for k in kv]
    b = Batch([L, L], kv, final, Hq, Hkv, D, page, seed=40)
    f = inv_freq(D)
    g = torch.Generator().manual_seed(41)
    qw, kw = ((0.2 * torch.randn(D, generator=g)).bfloat16() for _ in range(2))
    p = dg.head_params(Hq, Hkv, D, rope_steps=dg.rope_steps(f, DEV), q_weight=qw.to(DEV), k_weight=kw.to(DEV),
                       weight_offset=1.0)
    c = b.cache(kv)
    after = torch.zeros(2, dtype=torch.int32, device=DEV)
    read = dg.PagedCache(c.k, c.v, c.page_table, after, c.q_start)
    ws = dg.workspace(dg.paged_attn_workspace(b.T, Hq, c), DEV)
    for step in range(blocks):
        q, k, v = ((3 * torch.randn(b.T, h, D, generator=g)).bfloat16() for h in (Hq, Hkv, Hkv))
        pos = torch.cat([torch.arange(x, x + L, dtype=torch.int32) for x in kv])
        qd, kd, vd = q.to(DEV), k.to(DEV), v.to(DEV)
        qo, ko, out, enc = torch.empty_like(qd), torch.empty_like(kd), torch.empty_like(qd), torch.empty_like(qd)
        dg.qk_norm_rope(qd, kd, qo, ko, pos.to(DEV), p)
        dg.paged_attn(qo, c, out, b.scale, ws, k_new=ko, v_new=vd, causal=False)
        dg.paged_append(kd, vd, c, p, ws, kv_len_out=after)
        dg.paged_attn(qo, read, enc, b.scale, ws)
        torch.cuda.synchronize()
        status_ok(ws)
        close(qo, *norm_rope(q, pos, f, False, qw, 1e-6, 1.0))
        b.q, b.kn, b.vn, b.k, b.v = qo.cpu(), ko.cpu(), v, c.k.cpu(), c.v.cpu()
        close(out, *attention(b, False, 0, True, kv))
        now = [x + L for x in kv]
        assert after.tolist() == now
        for i in range(2):      # the appended keys are the canvas's own
            got, _ = b.keys(i, now[i])
            assert same_bits(got[kv[i]:], ko.cpu()[i * L:(i + 1) * L])
        close(enc, *attention(b, True, 0, False, now))
        c.kv_len.copy_(after)
        kv = now
