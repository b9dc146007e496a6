"""More GPU tests of the paged-cache operators: batches, layouts and values that are rare by themselves."""
import pytest
import torch

import block_diffusion_decoding_gb300 as dg
from tests._helpers import status_ok
from tests._paged import DEV, NAN, Batch, attention, close
from tests.test_gpu_paged import check_attn, run_attn, same_bits

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
