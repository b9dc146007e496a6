"""Inline PTX that reads or writes memory, by the sources: it is volatile and clobbers memory, so that the compiler
moves it neither over the wait for the kernel before nor over a barrier; or it is a load whose address is known behind
that wait alone."""
import os
import re

import pytest

from block_diffusion_decoding_gb300 import build as dgbuild

SOURCES = sorted(f for f in os.listdir(dgbuild.CSRC) if f.endswith((".cu", ".cuh", ".h")))
# PTX that reads or writes what the program's own loads and stores do, or orders it (tensor memory has no others, and a
# prefetch changes nothing)
MEMORY = re.compile(r"\s*(ld|st|atom|red|cp|mbarrier|griddepcontrol|barrier|fence|membar)\.")


def statements(text):
    """The asm statements of a source, comments and line breaks taken out."""
    text = re.sub(r"//[^\n]*", "", text)
    for m in re.finditer(r"\basm\b(\s+volatile)?\s*\(", text):
        depth, i, quoted = 1, m.end(), False
        while depth:
            c = text[i]
            if c == '"' and text[i - 1] != "\\":
                quoted = not quoted
            depth += 0 if quoted else (c == "(") - (c == ")")
            i += 1
        yield bool(m.group(1)), " ".join(text[m.start():i].split())


def test_the_reader_of_sources():
    got = list(statements('asm("ld.a(%0);" : "=r"(x)); // asm("st.b")\nasm volatile(\n"fence.x;" ::: "memory");'))
    assert got == [(False, 'asm("ld.a(%0);" : "=r"(x))'), (True, 'asm volatile( "fence.x;" ::: "memory")')]


@pytest.mark.parametrize("name", SOURCES)
def test_asm_that_touches_memory_says_so(name):
    with open(os.path.join(dgbuild.CSRC, name)) as f:
        text = f.read()
    found = [(v, s) for v, s in statements(text) if MEMORY.match(s.split('"')[1])]
    loose = [s for v, s in found if not v or '"memory"' not in s]
    # or the one address that it depends on comes out of an asm that does
    if loose and name == "dg_sample.cu":
        assert len(loose) == 1 and loose[0].startswith('asm("ld.global.nc.') and loose[0].endswith(': "l"(p))')
        assert set(re.findall(r"\bbase = ([a-z_]+)\(", text)) == {"behind_waits"} and "fetch<Stream>(base + first)" in text
        loose = []
    assert not loose, loose


def test_the_address_behind_the_waits():
    with open(os.path.join(dgbuild.CSRC, "dg_device.cuh")) as f:
        assert (True, 'asm volatile("" : "+l"(p) : : "memory")') in list(statements(f.read()))
