"""GPU tests of calls around drafted trees and the page pool that the operators' own tests leave out."""
import pytest
import torch

import block_diffusion_decoding_gb300 as dg
from tests import _trees
from tests._helpers import status_ok
from tests._paged import DEV, Batch, attention, close
from tests.test_gpu_pages import Pool
from tests.test_gpu_tree import i32

pytestmark = pytest.mark.gpu


def test_plan_reports_fewer_cached_tokens_than_nodes():
    """Nodes that the lengths are said to count, and do not: reported, positions from 0 on; the others' as ever."""
    n = [5, 3, 4]
    b = Batch(n, [9, 9, 9], [9, 9, 9], 1, 1, 128, 16)
    trees = [_trees.tree(m, 3 + i) for i, m in enumerate(n)]
    parents = i32([p for t in trees for p in t])
    ws = dg.workspace(dg.tree_plan_workspace(), DEV)
    for kv, bad in (([5, 9, 4], 0), ([4, 9, 4], 7), ([5, 9, 0], 7), ([0, 2, 3], 7)):
        c = b.cache(kv)
        mask, positions = torch.zeros(12, 1, dtype=torch.int32, device=DEV), i32([77] * 12)
        dg.tree_plan(parents, c, mask, ws, positions=positions, appended=True)
        assert dg.read_device_status(ws, clear=True) == bad, kv
        want, at = _trees.plan(trees, [max(k - m, 0) for k, m in zip(kv, n)], 1)
        assert torch.equal(mask.cpu(), _trees.as_int32(want)) and positions.tolist() == at, kv
        dg.tree_plan(parents, c, mask, ws, positions=positions)      # (not counted: all of these are lengths)
        status_ok(ws)


@pytest.mark.parametrize("kernel", ["single", "pair"])
@pytest.mark.parametrize("window", [0, 37])
@pytest.mark.parametrize("fresh", [False, True])
def test_chains_and_causal_attention_are_both_the_definition(monkeypatch, kernel, window, fresh):
    """A chain sees what causal attention of the same tokens sees: each operator is within its own bound of it, and so
    within both bounds of the other (not the same bits: one rounds its weights to one bf16 number, the other may keep
    two)."""
    monkeypatch.setenv("DG_PAGED_KERNEL", kernel)
    n, kv, D = [20, 3, 150], [333, 64, 90], 128
    stored = kv if fresh else [a + m for a, m in zip(kv, n)]
    b = Batch(n, stored, stored, 4, 2, D, 32, seed=8)
    rows, at = _trees.plan([_trees.tree(m, 0, chain=True) for m in n], kv, 5, window)
    c = b.cache(stored)
    ws = dg.workspace(dg.paged_tree_attn_workspace(b.T, 4, c), DEV)
    tree, causal = torch.zeros_like(b.q).to(DEV), torch.zeros_like(b.q).to(DEV)
    new = dict(k_new=b.kn.to(DEV), v_new=b.vn.to(DEV)) if fresh else {}
    dg.paged_tree_attn(b.q.to(DEV), c, tree, b.scale, ws, _trees.as_int32(rows).to(DEV), positions=i32(at), window=window, **new)
    dg.paged_attn(b.q.to(DEV), c, causal, b.scale, ws, causal=True, window=window, **new)
    status_ok(ws)
    want, bound = _trees.attention(b, rows, at, window, fresh, stored)
    also, also_bound = attention(b, True, window, fresh, stored)
    assert torch.equal(want, also) and torch.equal(bound, also_bound)
    close(tree, want, bound)
    close(causal, want, bound)


def test_forks_of_many_pages_of_several_layers():
    """More copies than the grid has blocks, each of many blocks' pieces, the last of them cut short: 320 forks of two
    prompts that end in a nearly full page of 1024 tokens, two layers."""
    p = Pool(322, 340, 3, 1024, layers=2, Hkv=1)
    kv = [1024 + 1003, 997] + [0] * 320
    p.check(p.reserve(kv))
    p.grow(kv)
    p.check(p.fork([b % 2 for b in range(320)], list(range(2, 322))))
    p.check(p.release(list(range(0, 322, 3))))
