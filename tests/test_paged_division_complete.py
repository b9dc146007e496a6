"""The parts that the paged attention's work is divided into are all of it: the tiles of every item add up, in the
order of the units, to all it has, and the unit named for an item's last part is the one that has it."""
import random
import subprocess

import pytest

from tests._paged_division import SOURCE, compile_to, run
from tests.test_paged_division import _case


def cases(seed, n, falling):
    """Ragged batches as in the other division test, and more of many query tiles; falling: row starts may decrease
    (the kernels then compute nothing, the walk alone does not know of it)."""
    rng = random.Random(seed)
    found = []
    while len(found) < n:
        c = _case(rng)
        if rng.random() < 0.3:      # whole items in turn, then a cut rest
            c[10:12] = [128, 256]
            c[9] = rng.choice([2, 76])
        T, B, Hkv, G = c[:4]
        start = c[12:12 + B + 1]
        if Hkv * (T * G // 128 + B) > 60000 or not falling and any(y < x for x, y in zip(start, start[1:])):
            continue
        found.append(c)
    return found


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    return compile_to(tmp_path_factory.mktemp("division"))


def test_on_the_host(program):
    n, rounds, cut = run(program, "host", cases(21, 800, False))
    assert n == 800 and rounds > 30 and cut > 2000, (n, rounds, cut)


def test_a_lost_tail_is_noticed(tmp_path):
    """The check itself: a walk that drops the last part of the items it cuts does not pass."""
    text = SOURCE.replace("parts.push_back(x);", "{ if (x.p.whole || x.p.t1 < x.p.nt) parts.push_back(x); }")
    assert text != SOURCE
    src = tmp_path / "lost"
    src.mkdir()
    import tests._paged_division as d
    old, d.SOURCE = d.SOURCE, text
    try:
        exe = compile_to(src)
    finally:
        d.SOURCE = old
    with pytest.raises(AssertionError, match="tiles"):
        run(exe, "host", cases(21, 100, False))
    assert subprocess.run([exe, "host"], input="", capture_output=True).returncode == 0


@pytest.mark.gpu
def test_on_the_device(program):
    n, rounds, cut = run(program, "device", cases(22, 1500, True))
    assert n == 1500 and rounds > 30 and cut > 2000, (n, rounds, cut)
