"""Loads from tensor memory are asynchronous: their registers hold nothing until
tcgen05.wait::ld, and only an operand keeps the compiler from moving a use of a
register ahead of an asm statement (a clobber of memory does not). The kernels'
sources are read for it: no machine that compiles them otherwise shows it."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "fp8_quantized_paged_store_gb300", "csrc")
SOURCES = {os.path.basename(p): open(p).read() for p in sorted(glob.glob(os.path.join(CSRC, "*.cu*")))}


def statements(text, instruction):
    return re.findall(r"asm volatile\(\s*\"" + re.escape(instruction) + r".*?\);", text, flags=re.S)


@pytest.mark.parametrize("name", list(SOURCES))
def test_every_wait_holds_the_loaded_registers(name):
    for s in statements(SOURCES[name], "tcgen05.wait::ld"):
        registers = re.findall(r'"\+r"\(r\[(\d+)\]\)', s)
        assert len(registers) in (16, 32) and [int(x) for x in registers] == list(range(len(registers)))


@pytest.mark.parametrize("name", list(SOURCES))
def test_every_load_is_followed_by_its_wait(name):
    """In the function that loads, or, by the function's name, in its caller,
    which then also ties the registers of further loads behind the same wait."""
    text = SOURCES[name]
    for f in re.findall(r"void (tmem_ld\w*)\((.*?)\n}", text, flags=re.S):
        if statements(f[1], "tcgen05.ld") and not f[0].endswith("_issue"):
            assert re.search(r"tmem_ld_wait\(r\);\s*$", f[1]), f[0]
    for issued in re.finditer(r"tmem_ld32_issue\([^;]*?, (\w+(?:\[\d\])?)\);", text):
        name_, behind = issued.group(1), text[issued.end():issued.end() + 200]
        tied = r"(tmem_ld_wait|after_wait)\(" + re.escape(name_) + r"\);"
        first = re.sub(r"\s*tmem_ld32_issue\([^;]*;", "", behind)
        assert re.match(r"(\s*(tmem_ld_wait|after_wait)\(\w+(\[\d\])?\);)*?\s*" + tied, first), issued.group(0)


def test_there_are_loads_to_check():
    assert sum(len(statements(t, "tcgen05.ld.")) for t in SOURCES.values()) >= 2
    assert sum(len(statements(t, "tcgen05.wait::ld")) for t in SOURCES.values()) >= 2
