"""Rows behind a tile's last one stay out of reach of the training epilogues, in
the gfx950 assembly the compiler writes for them.

A buffer descriptor bounds a tile's rows by the offset that the hardware compares
with its size: the lane's and the instruction's own.  A scalar offset comes on top
of that, unchecked.  So what reads or writes registers through a descriptor has no
scalar offset (the loads that write LDS have one, which counts along a row or down
the weights' k and never leaves the expert's weights or the row that the lane's
offset was checked for).  Runs on the CPU (hipcc cross-compiles)."""
import re

import pytest

from test_training_asm import assembly

ACCESS = re.compile(r"^buffer_(?:load|store)_\w+\s+(.*)$")
SCALAR = re.compile(r"s\[\d+:\d+\],\s*(\S+)")


def unchecked_offsets(asm):
    """(buffer accesses of registers seen, those with a scalar offset)"""
    seen, bad = 0, []
    for line in asm.split("\n"):
        t = line.split(";")[0].strip()
        m = ACCESS.match(t)
        if not m or m[1].split()[-1] == "lds":
            continue
        seen += 1
        if SCALAR.search(m[1])[1] != "0":
            bad.append(t)
    return seen, bad


def test_a_scalar_offset_is_seen():
    assert unchecked_offsets(" buffer_load_dwordx4 v[4:7], v1, s[0:3], s9 offen")[1]
    assert unchecked_offsets(" buffer_store_dword v4, v1, s[0:3], m0 offen offset:16")[1]
    assert unchecked_offsets(" buffer_store_dword v4, v1, s[0:3], 0 offen offset:16 ; s9") == (1, [])
    assert unchecked_offsets(" buffer_load_dwordx4 v1, s[0:3], s9 offen lds") == (0, [])


@pytest.mark.timeout(600)
def test_training_epilogues(tmp_path):
    seen, bad = unchecked_offsets(assembly("grouped_ffn.hip", tmp_path))
    assert seen, "no buffer accesses of registers: the pattern changed"
    assert not bad, f"{len(bad)} of {seen} with an unchecked offset, e.g. {bad[:3]}"
