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
