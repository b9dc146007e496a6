"""More GPU tests of the paged-cache operators: batches, layouts and values that are rare by themselves."""
import pytest
import torch

import block_diffusion_decoding_gb300 as dg
from tests._helpers import status_ok
from tests._paged import DEV, NAN, Batch, attention, close
from tests.test_gpu_paged import check_attn, kernel, run_attn, same_bits  # noqa: F401 (kernel: a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("causal,window,fresh", [(True, 0, False), (False, 0, True), (True, 60, True)])
@pytest.mark.parametrize("empty", [0, 4000])
def test_units_of_many_parts_at_head_dim_256(monkeypatch, causal, window, fresh, empty):
    """CTA pairs that take several items of one key tile each before a longer one, and with `empty` sequences
    of no new tokens between them, which make the walk over the parts the slowest role."""
    monkeypatch.setenv("DG_PAGED_KERNEL", "pair")
    g = torch.Generator().manual_seed(61)
    n, kv = [], []
    for i in range(420):
        long = i % 3 == 2
        n.append(1 if i % 5 else 3)
        kv.append(int(torch.randint(200, 401, (1,), generator=g)) if long else
                  int(torch.randint(1, 129, (1,), generator=g)))
        if empty and i % 60 == 59:
            n += [0] * (empty // 7)
            kv += [5] * (empty // 7)
    if not fresh:
        kv = [k + m for k, m in zip(kv, n)]
    check_attn(n, kv, 2, 2, 256, 16, causal, window, fresh, seed=62)


@pytest.mark.parametrize("D,window,fresh", [(128, 0, True), (256, 0, True), (128, 90, False), (256, 300, True)])
def test_hidden_values_in_every_border_tile(monkeypatch, D, window, fresh):
    """Units of several parts, all of whose border tiles hold values that some rows must not know of, in either
    CTA's half of the dims; in the next batch over the same workspace there are none.  The same bits every time."""
    monkeypatch.setenv("DG_PAGED_KERNEL", "pair")
    n, kv = [37 + 61 * (i % 5) for i in range(24)], [50 + 77 * (i % 7) for i in range(24)]
    if not fresh:
        kv = [k + m for k, m in zip(kv, n)]
    clean = Batch(n, kv, kv, 2, 2, D, 16, seed=63)
    b = Batch(n, kv, kv, 2, 2, D, 16, seed=63)
    for i in range(24):
        total = kv[i] + (n[i] if fresh else 0)
        for key in range(total - n[i] + 3, total, 29):     # seen by the rows from there on only
            for head in (0, 1):
                dim = (key * 7 + head) % (D // 2) + (D // 2 if (key + head) % 2 else 0)
                if key < kv[i]:
                    b.v[b.table[i, key // 16], key % 16, head, dim] = float("inf")
                else:
                    b.vn[int(b.q_start[i]) + key - kv[i], head, dim] = float("inf")
    want, bound = attention(b, True, window, fresh, kv)
    ws = dg.workspace(dg.paged_attn_workspace(b.T, 2, b.cache(kv)), DEV)
    first = None
    for turn in range(6):
        out = run_attn(b, True, window, fresh, kv, ws=ws)
        ends = torch.isinf(want)
        assert torch.equal(out.cpu().double()[ends], want[ends]) and ends.any()
        fine = torch.isfinite(want)
        assert ((out.cpu().double()[fine] - want[fine]).abs() <= bound[fine]).all()
        first = out if first is None else first
        assert same_bits(out, first)
        if turn == 0:
            close(run_attn(clean, True, window, fresh, kv, ws=ws), *attention(clean, True, window, fresh, kv))


@pytest.mark.parametrize("D,Hq", [(256, 8), (128, 16), (128, 2)])
def test_a_sequence_whose_values_have_overflowed_leaves_the_others_alone(monkeypatch, D, Hq):
    """One sequence of a decode batch, 40000 keys long, with nothing but NaN, or infinities, in its values: the
    others, whose parts the same CTAs work on, get the bits they get without it, and no wait runs out."""
    monkeypatch.setenv("DG_PAGED_KERNEL", "single")
    B, page, kv = 160, 64, 40000
    P = kv // page
    g = torch.Generator(device=DEV).manual_seed(71)
    k = torch.randn(2 * P, page, 1, D, generator=g, device=DEV, dtype=torch.bfloat16)
    v = torch.randn(2 * P, page, 1, D, generator=g, device=DEV, dtype=torch.bfloat16)
    table = torch.arange(P, device=DEV, dtype=torch.int32).repeat(B, 1)
    table[5] += P                               # the others share their pages
    c = dg.PagedCache(k, v, table, torch.full((B,), kv, device=DEV, dtype=torch.int32),
                      torch.arange(B + 1, device=DEV, dtype=torch.int32))
    q = torch.randn(B, Hq, D, generator=g, device=DEV, dtype=torch.bfloat16)
    ws = dg.workspace(dg.paged_attn_workspace(B, Hq, c), DEV)

    def run():
        out = torch.full_like(q, 5.0)
        dg.paged_attn(q, c, out, D ** -0.5, ws)
        status_ok(ws)
        return out

    clean = run()
    others = torch.arange(B, device=DEV) != 5
    good = v[P:].clone()
    inf = float("inf")
    for fill, want in ((NAN, NAN), (inf, inf), (-inf, -inf)):
        v[P:] = fill
        got = run()
        assert same_bits(got[others], clean[others])
        row = got[5].float()
        assert torch.isnan(row).all() if want != want else (row == want).all()
    v[P:] = inf
    v[P + 100, 7] = -inf
    assert torch.isnan(run()[5]).all()
    v[P:] = good
    v[P + 3, 9, 0, 5], v[2 * P - 1, 63, 0, D - 1], v[P, 0, 0, D - 1], v[P + 9, 1, 0, D // 2] = inf, inf, -inf, NAN
    got = run()
    keep = torch.ones(D, dtype=torch.bool, device=DEV)
    keep[[5, D // 2, D - 1]] = False
    assert same_bits(got[others], clean[others]) and same_bits(got[5][:, keep], clean[5][:, keep])
    assert (got[5][:, 5] == inf).all() and torch.isnan(got[5][:, [D // 2, D - 1]]).all()


@pytest.mark.parametrize("D,Hq,Hkv", [(128, 4, 1), (256, 2, 1), (128, 6, 3)])
@pytest.mark.parametrize("window,fresh", [(0, False), (0, True), (40, True)])
def test_infinite_values_that_some_tokens_of_a_few_see(kernel, D, Hq, Hkv, window, fresh):
    """Items of few rows but several tokens: infinities among the tokens' own values, which the earlier ones do
    not see, and among the cached ones; and a key that is infinite itself, whose value is too."""
    n, kv = [3, 2, 4, 1], [300, 7, 129, 500]
    if not fresh:
        kv = [k + m for k, m in zip(kv, n)]
    b = Batch(n, kv, kv, Hq, Hkv, D, 32, seed=64, strided=True)
    inf = float("inf")

    def put(s, back, dim, value, which="v"):
        """Into the key `back` before the last of sequence s."""
        key = kv[s] + (n[s] if fresh else 0) - 1 - back
        if key < kv[s]:
            (b.k if which == "k" else b.v)[b.table[s, key // 32], key % 32, 0, dim] = value
        else:
            (b.kn if which == "k" else b.vn)[int(b.q_start[s]) + key - kv[s], 0, dim] = value

    put(0, 0, 3, inf)
    put(0, 1, D - 1, -inf)
    put(0, 30, 17, inf)
    put(0, 2, 17, -inf)
    put(1, 1, D // 2, NAN)
    put(2, 0, 40, -inf)
    put(2, 3, 41, inf)
    put(3, 20, 9, inf)
    put(3, 20, 1, inf, "k")
    out = run_attn(b, True, window, fresh, kv).cpu().double()
    want, bound = attention(b, True, window, fresh, kv)
    # sequence 3's row has an infinite score: NaN, or (minus infinity) no weight, times an infinite value
    assert torch.equal(torch.isnan(out), torch.isnan(want)) and torch.isnan(want).any()
    ends = torch.isinf(want)
    assert torch.equal(out[ends], want[ends]) and ends.any()
    fine = torch.isfinite(want)
    assert torch.isfinite(out[fine]).all() and ((out[fine] - want[fine]).abs() <= bound[fine]).all()


@pytest.mark.parametrize("start,kv", [([-4, 2, 8], [14, 3]), ([0, 4, 90], [14, 3]), ([3, 6, 1000], [0, 20]),
                                      ([-10 ** 9, 8, 8], [5, 7]), ([0, 12, 12], [-3, 9]), ([0, 6, 2], [4, 9]),
                                      ([0, 4, 8], [2 ** 31 - 2, 1])])
def test_append_cuts_its_rows_as_the_attention_does(start, kv):
    """Row starts that leave the batch and lengths that cannot be: reported; the tokens there are lie where the
    attention looks for them, the new lengths count those, and a negative length stores nothing and stays."""
    T, page, cap = 12, 16, 48
    b = Batch([6, 6], [18, 30], [48, 48], 2, 1, 128, page, seed=65)
    c = b.cache(kv)
    c.q_start.copy_(torch.tensor(start, dtype=torch.int32))
    k0, v0 = c.k.cpu(), c.v.cpu()
    ws = dg.workspace(256, DEV)
    lens = torch.full((2,), 77, dtype=torch.int32, device=DEV)
    dg.paged_append(b.kn.to(DEV), b.vn.to(DEV), c, dg.head_params(2, 1, 128), ws, kv_len_out=lens)
    assert dg.read_device_status(ws, clear=True) == 7
    after = []
    for s in range(2):
        first = min(max(start[s], 0), T)
        end = max(min(start[s + 1], T), first)
        if kv[s] < 0:
            after.append(kv[s])
            continue
        after.append(min(kv[s] + end - first, 2 ** 31 - 1))
        for t in range(first, end):
            at = kv[s] + t - first
            if at < cap:
                k0[b.table[s, at // page], at % page] = b.kn[t]
                v0[b.table[s, at // page], at % page] = b.vn[t]
    assert lens.tolist() == after
    assert same_bits(c.k, k0) and same_bits(c.v, v0)


def test_page_layouts_that_are_dense_all_the_same():
    """Dimensions of one element have strides that say nothing: one kv head taken from a pool laid out by heads,
    a pool of one page.  They work; pools that are not dense are refused as before."""
    n, kv, page, D = [1, 5], [40, 17], 16, 128
    b = Batch(n, kv, kv, 4, 1, D, page, seed=66)
    want = run_attn(b, True, 0, False, kv)
    c = b.cache()
    by_head = [torch.empty(b.n_pages, 1, page, D, dtype=torch.bfloat16, device=DEV).copy_(t.transpose(1, 2))
               .transpose(1, 2) for t in (c.k, c.v)]
    by_head[0] = by_head[0].as_strided(by_head[0].shape, (page * D, D, 12345, 1))
    assert by_head[0].stride() != c.k.stride() and by_head[0].stride() != by_head[1].stride()
    ws = dg.workspace(dg.paged_attn_workspace(b.T, 4, c), DEV)
    out = torch.empty_like(b.q, device=DEV)
    dg.paged_attn(b.q.to(DEV), dg.PagedCache(*by_head, c.page_table, c.kv_len, c.q_start), out, b.scale, ws)
    status_ok(ws)
    assert same_bits(out, want)
    one = [t[2:3].as_strided((1, page, 1, D), (s, D, D, 1)) for t, s in ((c.k, 8), (c.v, 16 * D))]
    dg.PagedCache(*one, c.page_table, c.kv_len, c.q_start)
    for bad in ([c.k, c.v[::2]], [c.k, c.v.float()], [c.k[..., ::2], c.v[..., ::2]],
                [c.k[:, ::2], c.v[:, ::2]],
                [c.k[::2], c.v[:c.k[::2].shape[0]]], [c.k[:1].expand_as(c.k), c.v[:1].expand_as(c.v)]):
        with pytest.raises(dg.DgError):
            dg.PagedCache(*bad, c.page_table, c.kv_len, c.q_start)
    two = torch.empty(b.n_pages, 2, page, D, dtype=torch.bfloat16, device=DEV).transpose(1, 2)
    with pytest.raises(dg.DgError):      # two heads laid out by heads: not a token's row
        dg.PagedCache(two, two, c.page_table, c.kv_len, c.q_start)


@pytest.mark.parametrize("D,n,kv", [(128, [300], [5000]), (256, [300], [5000]), (128, [1], [9000]), (256, [3], [9000]),
                                    (128, [60], [4000]), (256, [64, 64], [3000, 4000])])
def test_workspace_of_the_queried_size_is_enough(kernel, D, n, kv):
    """Items cut between all the CTAs: nothing behind the workspace is written."""
    b = Batch(n, kv, kv, 4, 2, D, 64, seed=67)
    c = b.cache()
    need = dg.paged_attn_workspace(b.T, 4, c)
    room = dg.workspace(need + (1 << 20), DEV)
    room[need:] = 0xA5
    out = torch.empty_like(b.q, device=DEV)
    dg.paged_attn(b.q.to(DEV), c, out, b.scale, room[:need])
    status_ok(room)
    assert (room[need:] == 0xA5).all()
    close(out, *attention(b, True, 0, False, kv))
