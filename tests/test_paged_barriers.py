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
