"""How exact the trees' single-CTA attention is: it multiplies each softmax weight as two bf16 halves, as the other
paged attention of few rows does, so that verifying a drafted token is as exact as decoding it."""
import pytest
import torch

from tests import _trees
from tests._paged import Batch, close
from tests.test_paged_precision import WEIGHTS, split

CASES = [([1, 1], [40, 7], 4, 2, 128, 0, False), ([16], [300], 4, 1, 128, 0, False), ([5, 30], [20, 90], 4, 2, 128, 0, True),
         ([40, 9], [200, 33], 2, 1, 256, 0, False), ([64, 17], [250, 64], 4, 2, 128, 60, False),
         ([20], [90], 4, 4, 256, 30, True), ([150], [100], 2, 2, 128, 0, False)]


def case(n, kv, Hq, Hkv, D, window, fresh):
    """(batch, plan's rows and positions, stored tokens, (out, bound)): the definition, and a bound of the output's own
    rounding and of weights kept to WEIGHTS."""
    stored = kv if fresh else [a + m for a, m in zip(kv, n)]
    b = Batch(n, stored, stored, Hq, Hkv, D, 32, seed=17)
    rows, at = _trees.plan([_trees.tree(m, 5 + i) for i, m in enumerate(n)], kv, 5, window)
    out, bound = _trees.attention(b, rows, at, window, fresh, stored)
    size = (bound - 2 ** -8 * out.abs()) / (2 ** -8 + 2 ** -12)
    return b, rows, at, stored, (out, 2 ** -8 * out.abs() + WEIGHTS * size)


def test_the_bound_notices_one_half():
    """Weights as two halves keep to the bound, weights rounded to one bf16 do not."""
    g = torch.Generator().manual_seed(3)
    w = torch.rand(200, 12, generator=g)
    v = torch.randn(12, 64, generator=g).bfloat16().double()
    want = w.double() @ v / w.double().sum(1, keepdim=True)
    bound = 2 ** -8 * want.abs() + WEIGHTS * (w.double() @ v.abs()) / w.double().sum(1, keepdim=True)
    got = lambda p: (p.double() @ v / w.double().sum(1, keepdim=True)).bfloat16()  # noqa: E731
    close(got(split(w, torch.zeros_like(w, dtype=torch.bool))), want, bound)
    with pytest.raises(AssertionError, match="more than the bound"):
        close(got(w.bfloat16()), want, bound)


@pytest.mark.gpu
@pytest.mark.parametrize("n,kv,Hq,Hkv,D,window,fresh", CASES)
def test_single_kernel(monkeypatch, n, kv, Hq, Hkv, D, window, fresh):
    import block_diffusion_decoding_gb300 as dg
    from tests._helpers import status_ok

    monkeypatch.setenv("DG_PAGED_KERNEL", "single")
    b, rows, at, stored, (want, bound) = case(n, kv, Hq, Hkv, D, window, fresh)
    c = b.cache(stored)
    ws = dg.workspace(dg.paged_tree_attn_workspace(b.T, Hq, c), "cuda")
    out = torch.zeros_like(b.q).to("cuda")
    dg.paged_tree_attn(b.q.to("cuda"), c, out, b.scale, ws, _trees.as_int32(rows).to("cuda"),
                       positions=torch.tensor(at, dtype=torch.int32, device="cuda"), window=window,
                       **(dict(k_new=b.kn.to("cuda"), v_new=b.vn.to("cuda")) if fresh else {}))
    status_ok(ws)
    close(out, want, bound)
