"""GPU tests of calls around drafted trees and the page pool that the operators' own tests leave out."""
import pytest
import torch

import block_diffusion_decoding_gb300 as dg
from tests import _trees
from tests._helpers import status_ok
from tests._paged import DEV, Batch, close
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
