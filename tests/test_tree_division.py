"""The tree attention's work is divided into parts that are all of it, as the paged attention's: every key that a
node may see, at the depth of its index (further up a window's keys are earlier ones), is in one part of every item."""
import pytest

import tests._paged_division as division
from tests._paged_division import compile_to, run
from tests.test_paged_division_complete import cases


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    text = division.SOURCE.replace("PagedArgs", "PagedTreeArgs")
    old, division.SOURCE = division.SOURCE, text
    try:
        return compile_to(tmp_path_factory.mktemp("division"))
    finally:
        division.SOURCE = old


def trees(seed, n, falling):
    """The other test's batches; a node sees none behind it, so that every batch is a causal one."""
    return [c[:7] + [1] + c[8:] for c in cases(seed, n, falling)]


def test_on_the_host(program):
    n, rounds, cut = run(program, "host", trees(31, 800, False))
    assert n == 800 and rounds > 30 and cut > 2000, (n, rounds, cut)


@pytest.mark.gpu
def test_on_the_device(program):
    n, rounds, cut = run(program, "device", trees(32, 1500, True))
    assert n == 1500 and rounds > 30 and cut > 2000, (n, rounds, cut)
