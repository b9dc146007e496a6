"""The paged attention's workspace query: what the part slots of either kernel can hold, and no more."""
import ctypes

import pytest

import block_diffusion_decoding_gb300 as dg
from block_diffusion_decoding_gb300 import build as dgbuild

GOOD = 1 << 20
UNITS = 256     # CTAs that the query allows for


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("T,Hq,Hkv", [(0, 4, 2), (1, 4, 4), (5, 4, 2), (63, 4, 2), (64, 4, 2), (65, 4, 2), (9, 128, 1),
                                      (3000, 16, 8), (100000, 8, 8)])
def test_query_is_what_the_slots_take(D, T, Hq, Hkv):
    """Two parts of 128 rows for each CTA, or of 256 for each pair of them: a maximum and a sum, and D values in
    fp32, a row."""
    dgbuild.build()
    c = dg.PagedCacheArgs(GOOD, GOOD, GOOD, GOOD, GOOD, 0, 10, 16, 4, 2, Hkv, D)
    need = dg.lib().dg_paged_attn_workspace(T, Hq, ctypes.byref(c))
    folded = max(T, 1) * Hq // Hkv
    parts = max(2 * UNITS * min(128, folded), 2 * (UNITS // 2) * min(256, folded))
    least = 256 + UNITS * 32 + parts * (8 + 4 * D)
    assert least <= need <= least + 2 * 256
