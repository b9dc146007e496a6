"""The barriers of the paged attention kernels, read from their source: which waits could miss a phase."""
import os
import re

import pytest

from block_diffusion_decoding_gb300 import build as dgbuild

FILES = ("dg_paged_pair.cu", "dg_paged_attn.cu", "dg_paged.cuh")


def source(name):
    with open(os.path.join(dgbuild.CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def waits(text):
    """(barrier, parity) of every wait, as they are written."""
    calls = re.findall(r"mbar_wait(?:_poll)?(?:<[^>]*>)?\(\s*&?((?:[^,()]|\([^()]*\))+),\s*((?:[^,()]|\((?:[^()]|\([^()]*\))*\))+),", text)
    return [(re.sub(r"\[.*", "", b.strip()).replace("sh.", ""), p.strip()) for b, p in calls]


@pytest.mark.parametrize("name", FILES)
def test_a_wait_for_a_fixed_phase_is_on_a_barrier_that_is_used_once(name):
    """A parity names a phase and every second one after it: a wait for a given parity is safe only on a barrier
    that completes one phase in all, or where the phases are counted.  A barrier waited for in both ways is used
    again, and the fixed wait may find it two phases on, where it blocks until the third."""
    found = waits(source(name))
    assert found
    fixed = {b for b, p in found if p.isdigit()}
    counted = {b for b, p in found if not p.isdigit()}
    assert not fixed & counted, fixed & counted


def test_tiles_that_land_on_both_ctas_are_released_to_the_products():
    """Where a V half lands on its own CTA's barrier, the arrival of P is the only sign to the even CTA's products
    that the other half is there and clean, and that a value was zeroed: it has to release memory, in the odd CTA
    and wherever a word was stored to the other one, at cluster scope."""
    text = source("dg_paged_pair.cu")
    landed = text[text.index("mbar_wait_poll(&sh.v_land[vs]"):]
    tile = landed[:landed.index("} else {")]
    assert "sh.p_full" in tile and "st_cluster(" in tile
    assert "mbar_arrive_cluster(lead_of(&sh.p_full" in tile
    assert "relaxed" not in tile
    local = re.search(r"if \(([^()]*)\) mbar_arrive\(&sh\.p_full", tile)
    assert local is None or local.group(1) == "r == 0 && !hid"
    # the words stored to the other CTA are read behind a wait that acquires at that scope
    assert "mbar_wait_poll<true>(&sh.o_full" in text
