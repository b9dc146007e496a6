"""GPU tests of the drafted trees' operators against their definitions: dg_tree_plan, dg_paged_tree_attn and
dg_paged_tree_commit, alone and as a server verifies drafts with them."""
import random

import pytest
import torch

import block_diffusion_decoding_gb300 as dg
from tests import _trees
from tests._helpers import status_ok
from tests._paged import DEV, NAN, Batch, close

pytestmark = pytest.mark.gpu


def same_bits(a, b):
    return torch.equal(a.contiguous().view(torch.int16).cpu(), b.contiguous().view(torch.int16).cpu())


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


# ---------------------------------------------------------------- plan
@pytest.mark.parametrize("n,words,window,appended,pad,chain", [
    ([1], 1, 0, False, 0, False),
    ([0, 1, 0, 32], 1, 0, False, 3, False),
    ([33, 5, 64, 31], 2, 0, True, 0, False),
    ([64, 17, 40], 3, 4, False, 1, False),
    ([300], 10, 0, True, 0, True),
    ([300, 2], 10, 7, False, 0, True),
    ([1000, 1, 4096, 129], 128, 0, False, 2, False),
    ([7] * 700, 1, 1, False, 0, False),
])
def test_plan(n, words, window, appended, pad, chain):
    r = random.Random(1)
    trees = [_trees.tree(m, 5 + i, chain=chain) for i, m in enumerate(n)]
    kv = [r.randrange(0, 500) + (m if appended else 0) for m in n]
    b = Batch(n, [1] * len(n), [1] * len(n), 1, 1, 128, 16, pad=pad)
    T = b.T
    table = torch.zeros(len(n), 512, dtype=torch.int32, device=DEV)
    c = dg.PagedCache(b.k.to(DEV), b.v.to(DEV), table, i32(kv), b.q_start.to(DEV))
    mask, positions = torch.full((T, words), 77, dtype=torch.int32, device=DEV), torch.full((T,), 77, dtype=torch.int32, device=DEV)
    ws = dg.workspace(dg.tree_plan_workspace(), DEV)
    parents = i32([p for t in trees for p in t] + [5] * pad)
    dg.tree_plan(parents, c, mask, ws, positions=positions, window=window, appended=appended)
    status_ok(ws)
    base = [k - m if appended else k for k, m in zip(kv, n)]
    want, at = _trees.plan(trees, base, words, window)
    rows = sum(n)
    assert torch.equal(mask[:rows].cpu(), _trees.as_int32(want))
    assert positions[:rows].tolist() == at
    assert (mask[rows:] == 77).all() and (positions[rows:] == 77).all()
    again = torch.full((T, words), 77, dtype=torch.int32, device=DEV)
    dg.tree_plan(parents, c, again, ws, window=window)           # no positions
    assert torch.equal(mask, again)


def test_plan_reports_what_is_no_tree():
    """A parent that is not lower than its node, one below -1, a node past the mask, rows that leave the batch."""
    b = Batch([4, 40], [3, 3], [3, 3], 1, 1, 128, 16)
    ws = dg.workspace(256, DEV)
    c = b.cache([3, 3])
    good = _trees.tree(4, 1) + _trees.tree(40, 2)
    for change in ((2, 2), (1, 3), (3, -2), (3, 900)):
        parents = list(good)
        parents[change[0]] = change[1]
        mask = torch.zeros(44, 2, dtype=torch.int32, device=DEV)
        dg.tree_plan(i32(parents), c, mask, ws)
        assert dg.read_device_status(ws, clear=True) == 7
        parents[change[0]] = -1
        want, _ = _trees.plan([parents[:4], parents[4:]], [3, 3], 2)
        assert torch.equal(mask.cpu(), _trees.as_int32(want))
    mask = torch.zeros(44, 1, dtype=torch.int32, device=DEV)     # 40 nodes in 32 bits
    dg.tree_plan(i32(good), c, mask, ws)
    assert dg.read_device_status(ws, clear=True) == 7
    want, _ = _trees.plan([good[:4], good[4:]], [3, 3], 1)
    assert torch.equal(mask.cpu(), _trees.as_int32(want))
    for start in ([0, 4, 99], [-3, 4, 44], [0, 30, 20], [0, 4, 44]):
        c.q_start.copy_(torch.tensor(start, dtype=torch.int32))
        dg.tree_plan(i32(good), c, torch.zeros(44, 2, dtype=torch.int32, device=DEV), ws)
        assert dg.read_device_status(ws, clear=True) == (0 if start == [0, 4, 44] else 7)


# ---------------------------------------------------------------- attention
def check_attn(n, kv, Hq, Hkv, D, page, window=0, fresh=False, pad=0, strided=False, words=None, chain=False, seed=0,
               mask=None):
    total = [a + m for a, m in zip(kv, n)]
    b = Batch(n, kv if fresh else total, kv if fresh else total, Hq, Hkv, D, page, seed=seed, pad=pad, strided=strided)
    trees = [_trees.tree(m, seed + i, chain=chain) for i, m in enumerate(n)]
    words = max(1, -(-max(n) // 32)) if words is None else words
    rows, at = _trees.plan(trees, kv, words, window)
    if mask is not None:
        rows = mask(rows)
    T = sum(n)
    bits = torch.zeros(b.T, words, dtype=torch.int32)
    bits[:T] = _trees.as_int32(rows)
    bits[T:] = -1
    pos = torch.full((b.T,), -5, dtype=torch.int32)
    pos[:T] = torch.tensor(at, dtype=torch.int32)
    c = b.cache(kv if fresh else total)
    ws = dg.workspace(dg.paged_tree_attn_workspace(b.T, Hq, c), DEV)
    out = b.rows(torch.full_like(b.q, 5.0))
    dg.paged_tree_attn(b.rows(b.q), c, out, b.scale, ws, bits.to(DEV), k_new=b.rows(b.kn) if fresh else None,
                       v_new=b.rows(b.vn) if fresh else None, positions=pos.to(DEV) if window else None, window=window)
    torch.cuda.synchronize()
    status_ok(ws)
    want, bound = _trees.attention(b, rows, at, window, fresh, kv if fresh else total)
    close(out[:T], want[:T], bound[:T])
    assert (out[T:] == 5.0).all()
    return out


@pytest.mark.parametrize("kernel", ["single", "pair"])
@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("n,kv,Hq,Hkv,page,window,fresh,pad", [
    ([1], [0], 1, 1, 16, 0, False, 0),
    ([1], [0], 4, 1, 16, 0, True, 0),
    ([16], [300], 4, 1, 16, 0, False, 0),
    ([5, 0, 33, 1], [20, 7, 0, 129], 4, 2, 48, 0, False, 2),
    ([5, 0, 33, 1], [20, 7, 0, 129], 4, 2, 48, 0, True, 2),
    ([64, 17], [1000, 63], 2, 1, 64, 0, False, 0),
    ([64, 17], [1000, 64], 2, 1, 64, 100, False, 0),
    ([64, 17], [1000, 3], 3, 1, 32, 40, True, 0),
    ([200, 3], [130, 500], 2, 2, 128, 0, True, 1),
    ([200, 3], [131, 500], 2, 2, 128, 16, False, 1),
    ([3], [250], 8, 1, 16, 1, True, 0),
])
def test_attn(monkeypatch, kernel, D, n, kv, Hq, Hkv, page, window, fresh, pad):
    monkeypatch.setenv("DG_PAGED_KERNEL", kernel)
    check_attn(n, kv, Hq, Hkv, D, page, window, fresh, pad)


@pytest.mark.parametrize("kernel", ["single", "pair"])
def test_attn_strides_and_wide_masks(monkeypatch, kernel):
    monkeypatch.setenv("DG_PAGED_KERNEL", kernel)
    check_attn([40, 9], [77, 200], 4, 2, 128, 32, strided=True, words=7)
    check_attn([40, 9], [77, 200], 4, 2, 256, 32, fresh=True, strided=True, words=128)
    check_attn([70], [33], 2, 1, 128, 16, words=1)               # nodes past the mask: seen by nobody


@pytest.mark.parametrize("kernel", ["single", "pair"])
@pytest.mark.parametrize("fresh", [False, True])
def test_attn_rows_that_see_nothing_and_bits_of_nobody(monkeypatch, kernel, fresh):
    """No cached key and no bit: zeros; bits of later nodes and past the tree's mean nothing; of the others any
    pattern is taken."""
    monkeypatch.setenv("DG_PAGED_KERNEL", kernel)
    out = check_attn([6, 50], [0, 0], 4, 2, 128, 16, fresh=fresh, words=2,
                     mask=lambda rows: [[0, 0] if i % 3 == 0 else [x | 0xFFFFFFC0 if i < 6 else x, 0xFFFFFFFF if i < 6 else y]
                                        for i, (x, y) in enumerate(rows)])
    assert (out[0] == 0).all() and (out[3] == 0).all()
    r = random.Random(3)
    check_attn([90, 31], [5, 140], 2, 1, 128, 16, fresh=fresh, mask=lambda rows: [[r.getrandbits(32) for _ in x] for x in rows])


def test_attn_is_causal_attention_for_chains():
    """A chain sees what causal attention of the same tokens sees: the same kernels' arithmetic, the same bits."""
    for fresh in (False, True):
        for window in (0, 37):
            n, kv, D = [20, 3], [333, 64], 128
            total = [a + m for a, m in zip(kv, n)]
            b = Batch(n, kv if fresh else total, kv if fresh else total, 4, 2, D, 32, seed=8)
            rows, at = _trees.plan([_trees.tree(m, 0, chain=True) for m in n], kv, 1, window)
            c = b.cache(kv if fresh else total)
            ws = dg.workspace(dg.paged_tree_attn_workspace(b.T, 4, c), DEV)
            got, want = torch.zeros_like(b.q).to(DEV), torch.zeros_like(b.q).to(DEV)
            new = dict(k_new=b.kn.to(DEV), v_new=b.vn.to(DEV)) if fresh else {}
            dg.paged_tree_attn(b.q.to(DEV), c, got, b.scale, ws, _trees.as_int32(rows).to(DEV), positions=i32(at),
                               window=window, **new)
            dg.paged_attn(b.q.to(DEV), c, want, b.scale, ws, causal=True, window=window, **new)
            assert (got.float() - want.float()).abs().max() <= 2 ** -6   # (parts are cut elsewhere)
            status_ok(ws)


@pytest.mark.parametrize("kernel", ["single", "pair"])
@pytest.mark.parametrize("fresh", [False, True])
@pytest.mark.parametrize("D", [128, 256])
def test_attn_values_that_are_not_finite_reach_only_those_who_see_them(monkeypatch, kernel, fresh, D):
    """An infinite value of one node reaches its descendants' rows in its dimension, nobody else's."""
    monkeypatch.setenv("DG_PAGED_KERNEL", kernel)
    n, kv = [40], [100]
    b = Batch(n, kv if fresh else [140], kv if fresh else [140], 2, 1, D, 16, seed=4)
    parents = _trees.tree(40, 9)
    rows, at = _trees.plan([parents], kv, 2)
    bad = 17
    if fresh:
        b.vn[bad, 0, 5] = float("inf")
    else:
        place = 100 + bad
        b.v[b.table[0, place // 16], place % 16, 0, 5] = float("inf")
    c = b.cache()
    ws = dg.workspace(dg.paged_tree_attn_workspace(40, 2, c), DEV)
    out = torch.zeros_like(b.q).to(DEV)
    dg.paged_tree_attn(b.q.to(DEV), c, out, b.scale, ws, _trees.as_int32(rows).to(DEV),
                       k_new=b.kn.to(DEV) if fresh else None, v_new=b.vn.to(DEV) if fresh else None)
    status_ok(ws)
    out = out.cpu()
    sees = torch.tensor([x[bad // 32] >> bad % 32 & 1 for x in rows], dtype=torch.bool)
    assert 0 < sees.sum() < 40
    assert torch.isinf(out[sees][..., 5]).all()
    fine = torch.isfinite(out)
    fine[sees, :, 5] = True
    assert fine.all()
    b.vn[torch.isinf(b.vn)] = 0
    b.v[torch.isinf(b.v)] = 0
    want, bound = _trees.attention(b, rows, at, 0, fresh, kv if fresh else [140])
    close(out[~sees], want[~sees], bound[~sees])


def test_attn_batches_of_many_items():
    """Items that are cut, whole items of several rounds, and single tokens among them."""
    r = random.Random(2)
    n = [r.choice([0, 1, 7, 30, 64]) for _ in range(40)]
    kv = [r.choice([0, 5, 600, 900]) for _ in n]
    check_attn(n, kv, 4, 2, 128, 64, seed=3)
    check_attn([300, 20], [700, 900], 4, 2, 128, 64, window=200, fresh=True, seed=3)


def test_attn_positions_outside_the_tree_are_cut():
    n, kv, window = [6], [50], 20
    b = Batch(n, [56], [56], 2, 1, 128, 16, seed=5)
    rows, at = _trees.plan([_trees.tree(6, 1)], kv, 1, window)
    c = b.cache()
    ws = dg.workspace(dg.paged_tree_attn_workspace(6, 2, c), DEV)
    outs = []
    for pos in ([-2 ** 31, 49, 50, 55, 56, 2 ** 31 - 1], [50, 50, 50, 55, 55, 55]):
        out = torch.zeros_like(b.q).to(DEV)
        dg.paged_tree_attn(b.q.to(DEV), c, out, b.scale, ws, _trees.as_int32(rows).to(DEV), positions=i32(pos), window=window)
        outs.append(out)
    status_ok(ws)
    assert same_bits(*outs)


# ---------------------------------------------------------------- commit
def commit_case(n, kv, Hkv, D, page, layers, path_max, seed, pad=0, interleaved=False, accept=0.8):
    r = random.Random(seed)
    total = [a + m for a, m in zip(kv, n)]
    b = Batch(n, total, total, Hkv, Hkv, D, page, seed=seed, pad=pad)
    g = torch.Generator().manual_seed(seed)
    shape = (layers, b.n_pages, page, Hkv, D)
    k, v = (torch.randn(shape, generator=g).bfloat16() for _ in range(2))
    trees = [_trees.tree(m, seed + i) for i, m in enumerate(n)]
    tokens = [[r.randrange(3) for _ in t] for t in trees]        # siblings with equal tokens among them
    sampled = [[r.randrange(3) if r.random() < accept else 9 for _ in t] for t in trees]
    kd, vd = k.to(DEV), v.to(DEV)
    if interleaved:                                              # the layers of a page side by side
        wide = torch.zeros(b.n_pages, 2, layers, page, Hkv, D, dtype=torch.bfloat16, device=DEV)
        wide[:, 0], wide[:, 1] = kd.transpose(0, 1), vd.transpose(0, 1)
        kd, vd = wide[:, 0].transpose(0, 1), wide[:, 1].transpose(0, 1)
    c = dg.PagedCache(kd[0], vd[0], b.table.to(DEV), i32(total), b.q_start.to(DEV))
    flat = lambda x: i32([y for t in x for y in t] + [0] * pad)  # noqa: E731
    out = [torch.full((len(n), path_max), 55, dtype=torch.int32, device=DEV)] + [torch.full((len(n),), 55, dtype=torch.int32, device=DEV) for _ in range(3)]
    ws = dg.workspace(dg.paged_tree_commit_workspace(), DEV)
    return b, k, v, kd, vd, c, trees, tokens, sampled, flat, out, ws, total


@pytest.mark.parametrize("n,kv,Hkv,D,page,layers,path_max,pad,interleaved", [
    ([1], [0], 1, 128, 16, 1, 4, 0, False),
    ([16], [300], 1, 128, 16, 2, 16, 0, False),
    ([0, 33, 1, 64], [5, 13, 0, 100], 2, 128, 48, 3, 16, 2, False),
    ([40, 7, 200], [60, 31, 5], 8, 256, 32, 2, 3, 0, True),
    ([40, 7, 200], [60, 31, 5], 5, 128, 16, 4, 150, 1, True),
    ([64] * 50, [17 * i for i in range(50)], 2, 128, 64, 2, 8, 0, False),
])
def test_commit(n, kv, Hkv, D, page, layers, path_max, pad, interleaved):
    b, k, v, kd, vd, c, trees, tokens, sampled, flat, out, ws, total = commit_case(n, kv, Hkv, D, page, layers, path_max, 3, pad, interleaved)
    dg.paged_tree_commit(flat(tokens), flat(trees), flat(sampled), c, *out, ws, layers=(kd, vd))
    status_ok(ws)
    moved = 0
    for s, t in enumerate(trees):
        path, nxt = _trees.walk(t, tokens[s], sampled[s], path_max)
        assert out[0][s].tolist() == path + [0] * (path_max - len(path))
        assert out[1][s].item() == len(path) and out[2][s].item() == nxt
        assert out[3][s].item() == kv[s] + len(path)
        places = [(b.table[s, x // page].item(), x % page) for x in range(total[s])]
        for pool in (k, v):
            rows = [pool[:, places[kv[s] + i][0], places[kv[s] + i][1]].clone() for i in path]
            for j, row in enumerate(rows):
                pool[:, places[kv[s] + j][0], places[kv[s] + j][1]] = row
        moved += sum(i != j for j, i in enumerate(path))
    assert same_bits(kd, k) and same_bits(vd, v)                 # every other byte as it was
    assert moved > 0 or len(n) == 1


def test_commit_long_paths():
    """A path longer than a block's turn; one layer without `layers`."""
    n, kv = [400], [21]
    b, k, v, kd, vd, c, trees, tokens, sampled, flat, out, ws, total = commit_case(n, kv, 1, 128, 32, 1, 380, 4)
    trees = [[-1, 0] + list(range(1, 399))]
    trees[0][2] = 0                                              # node 1 is passed by: everything moves
    tokens, sampled = [[7] * 400], [[7] * 400]
    tokens[0][1] = 8
    dg.paged_tree_commit(flat(tokens), flat(trees), flat(sampled), c, *out, ws)
    status_ok(ws)
    path = [0] + list(range(2, 381))
    assert out[0][0].tolist() == path and out[3].tolist() == [21 + 380] and out[2].tolist() == [7]
    places = [(b.table[0, x // 32].item(), x % 32) for x in range(421)]
    rows = [k[0, places[21 + i][0], places[21 + i][1]].clone() for i in path]
    for j, row in enumerate(rows):
        k[0, places[21 + j][0], places[21 + j][1]] = row
    assert same_bits(kd, k)


def test_commit_reports_what_it_cannot_do():
    b, k, v, kd, vd, c, trees, tokens, sampled, flat, out, ws, total = commit_case([20, 30], [10, 40], 1, 128, 16, 2, 16, 6)
    before = kd.clone()
    c.kv_len.copy_(torch.tensor([5, 70]))                        # fewer cached tokens than nodes
    dg.paged_tree_commit(flat(tokens), flat(trees), flat(sampled), c, *out, ws, layers=(kd, vd))
    assert dg.read_device_status(ws, clear=True) == 7
    assert out[1][0].item() == 0 and out[2][0].item() == -1 and out[3][0].item() == 5
    first = b.table[0, :2].long()
    assert same_bits(kd[:, first], before[:, first])
    # pages that do not exist: nothing is written to them, nothing else is touched
    b, k, v, kd, vd, c, trees, tokens, sampled, flat, out, ws, total = commit_case([30], [40], 1, 128, 16, 2, 16, 6)
    trees = [[-1, 0, 0] + list(range(2, 29))]                    # everything behind node 1 moves
    tokens, sampled = [[7, 8] + [7] * 28], [[7] * 30]
    c.page_table.copy_(torch.full_like(c.page_table, 10 ** 6))
    before = kd.clone()
    dg.paged_tree_commit(flat(tokens), flat(trees), flat(sampled), c, *out, ws, layers=(kd, vd))
    path, _ = _trees.walk(trees[0], tokens[0], sampled[0], 16)
    assert path != list(range(len(path)))
    assert dg.read_device_status(ws, clear=True) == 7 and same_bits(kd, before)


# ---------------------------------------------------------------- a step of verification, as a server runs it
def test_verification_step_in_a_graph():
    """Reserve, plan, append at the plan's positions, attend, draw, commit: captured once, replayed with other
    drafts, against the same steps done by hand."""
    r = random.Random(11)
    B, n, Hq, Hkv, D, page, V, layers, path_max = 3, 12, 4, 2, 128, 16, 500, 2, 6
    kv = [30, 0, 47]
    n_pages = 40
    g = torch.Generator().manual_seed(2)
    k, v = (torch.randn(layers, n_pages, page, Hkv, D, generator=g).bfloat16().to(DEV) for _ in range(2))
    table = torch.full((B, 8), -1, dtype=torch.int32)
    order = torch.randperm(n_pages, generator=g).int()
    at, refs = 0, torch.zeros(n_pages, dtype=torch.int32)
    for s in range(B):
        m = -(-kv[s] // page)
        table[s, :m] = order[at:at + m]
        refs[order[at:at + m].long()] = 1
        at += m
    free = torch.zeros(n_pages, dtype=torch.int32)
    free[:n_pages - at] = order[at:]
    q_start = i32([0, n, 2 * n, 3 * n])
    table, lens, after = table.to(DEV), i32(kv), i32([0] * B)
    before = [dg.PagedCache(k[x], v[x], table, lens, q_start) for x in range(layers)]
    behind = [dg.PagedCache(k[x], v[x], table, after, q_start) for x in range(layers)]
    pool = dg.PagePool(before[0], free.to(DEV), i32([n_pages - at]), refs.to(DEV))
    T = B * n
    parents, tokens = (torch.zeros(T, dtype=torch.int32, device=DEV) for _ in range(2))
    mask, positions = torch.zeros(T, 1, dtype=torch.int32, device=DEV), torch.zeros(T, dtype=torch.int32, device=DEV)
    q, kn, vn = (torch.zeros(layers, T, h, D, dtype=torch.bfloat16, device=DEV) for h in (Hq, Hkv, Hkv))
    out = torch.zeros_like(q)
    logits, u = torch.zeros(T, V, dtype=torch.bfloat16, device=DEV), torch.zeros(T, device=DEV)
    temp, sampled = torch.full((T,), 0.7, device=DEV), torch.zeros(T, dtype=torch.int32, device=DEV)
    path, n_path, nxt = torch.zeros(B, path_max, dtype=torch.int32, device=DEV), i32([0] * B), i32([0] * B)
    heads = dg.head_params(Hq, Hkv, D)
    ws = dg.workspace(dg.paged_tree_attn_workspace(T, Hq, before[0]), DEV)
    stream = torch.cuda.Stream()

    def step():
        dg.paged_reserve(pool, ws)
        dg.tree_plan(parents, before[0], mask, ws, positions=positions)
        for x in range(layers):
            dg.paged_append(kn[x], vn[x], before[x], heads, ws, positions=positions, kv_len_out=after)
            dg.paged_tree_attn(q[x], behind[x], out[x], D ** -0.5, ws, mask)
        dg.sample_logits(logits, sampled, u, temperature=temp)
        dg.paged_tree_commit(tokens, parents, sampled, behind[0], path, n_path, nxt, lens, ws, layers=(k, v))

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        step()
    want = [[[k[x, table[s, j // page].item(), j % page].clone() for j in range(kv[s])] for s in range(B)] for x in range(layers)]
    wantv = [[[v[x, table[s, j // page].item(), j % page].clone() for j in range(kv[s])] for s in range(B)] for x in range(layers)]
    for turn in range(3):
        trees = [_trees.tree(n, 100 * turn + s, back=3) for s in range(B)]
        toks = [[r.randrange(V) for _ in range(n)] for _ in range(B)]
        parents.copy_(i32([p for t in trees for p in t]))
        tokens.copy_(i32([x for t in toks for x in t]))
        for dst in (q, kn, vn):
            dst.copy_(torch.randn(dst.shape, generator=g).bfloat16())
        # each node's logits are sure of one of its children
        x = torch.zeros(T, V)
        for s in range(B):
            for i in range(n):
                kids = [c for c in range(n) if trees[s][c] == i]
                x[s * n + i, toks[s][r.choice(kids)] if kids and r.random() < 0.8 else r.randrange(V)] = 60
        logits.copy_(x.bfloat16())
        u.copy_(torch.rand(T, generator=g))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        status_ok(ws)
        got = sampled.tolist()
        assert got == x.argmax(1).tolist()
        for s in range(B):
            p, end = _trees.walk(trees[s], toks[s], got[s * n:(s + 1) * n], path_max)
            rows, pos = _trees.plan([trees[s]], [len(want[0][s])], 1)
            for layer in range(layers):
                keys = torch.stack(want[layer][s] + list(kn[layer, s * n:(s + 1) * n])).cpu()
                vals = torch.stack(wantv[layer][s] + list(vn[layer, s * n:(s + 1) * n])).cpu()
                base = keys.shape[0] - n
                for i in range(n):
                    seen = list(range(base)) + [base + j for j in range(n) if rows[i][0] >> j & 1]
                    for h in range(Hq):
                        w = torch.softmax(keys[seen, h // 2].double() @ q[layer, s * n + i, h].double().cpu() * D ** -0.5, 0)
                        o = w @ vals[seen, h // 2].double()
                        bound = 2 ** -8 * o.abs() + (2 ** -8 + 2 ** -12) * (w @ vals[seen, h // 2].double().abs())
                        close(out[layer, s * n + i, h], o, bound)
                want[layer][s] += [kn[layer, s * n + i].clone() for i in p]
                wantv[layer][s] += [vn[layer, s * n + i].clone() for i in p]
            assert path[s].tolist()[:len(p)] == p and n_path[s].item() == len(p) and nxt[s].item() == end
            assert lens[s].item() == len(want[0][s])
            for layer in range(layers):
                for j, row in enumerate(want[layer][s]):
                    assert same_bits(k[layer, table[s, j // page].item(), j % page], row)
    held = [p for s in range(B) for p in table[s, :-(-(lens[s].item() + n) // page)].tolist()]
    assert len(set(held)) == len(held)


def test_plan_follows_a_long_chain_for_4096_nodes():
    """A chain that no mask has room for, as a prompt beside trees would be, ends soon, and is reported."""
    n = 5000
    b = Batch([n], [1], [1], 1, 1, 128, 16)
    c = dg.PagedCache(b.k.to(DEV), b.v.to(DEV), torch.zeros(1, 512, dtype=torch.int32, device=DEV), i32([9]), b.q_start.to(DEV))
    mask, positions = torch.zeros(n, 128, dtype=torch.int32, device=DEV), torch.zeros(n, dtype=torch.int32, device=DEV)
    ws = dg.workspace(dg.tree_plan_workspace(), DEV)
    dg.tree_plan(i32(range(-1, n - 1)), c, mask, ws, positions=positions)
    assert dg.read_device_status(ws, clear=True) == 7
    assert positions.tolist() == [9 + min(i, 4095) for i in range(n)]
    want, _ = _trees.plan([list(range(-1, 4095))], [9], 128)
    assert torch.equal(mask[:4096].cpu(), _trees.as_int32(want))
