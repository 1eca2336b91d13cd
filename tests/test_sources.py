"""What the CUDA sources must not hold (CPU only)."""
import glob
import os
import re

import pytest

from w4a16_linear_layers_gb300 import build as qbuild

SOURCES = sorted(p for ext in ("cu", "cuh", "cpp", "h") for p in glob.glob(os.path.join(qbuild.CSRC, "*." + ext)))

# an instruction in the inline assembly: its mnemonic, up to the operands or
# the end of the statement, its neighbouring literals joined
STATEMENT = re.compile(r'"((?:[^"\\]|\\.)*)"')
SPREAD = "multi" + "cast"


def bulk_copies(text):
    """The bulk-copy instructions (tiled or plain) of a source's inline assembly."""
    joined = re.sub(r'"\s*\n\s*"', "", text)
    return [i for lit in STATEMENT.findall(joined) for i in re.split(r"\\n|;", lit) if "cp.async.bulk" in i]


def test_the_search_sees_an_instruction_over_two_literals():
    text = 'asm volatile(\n  "cp.async.bulk.tensor.2d.shared::cluster.global.tile"\n  ".%s::cluster [%%0], [%%1];" ::);' % SPREAD
    assert [SPREAD in i for i in bulk_copies(text)] == [True]


@pytest.mark.parametrize("path", SOURCES, ids=os.path.basename)
def test_no_copy_goes_to_several_blocks(path):
    """A copy that lands in several blocks' shared memory must not read a
    peer's memory, and the library also runs where there are peers."""
    with open(path) as f:
        assert [i for i in bulk_copies(f.read()) if SPREAD in i] == []


def test_the_copies_are_found():
    found = []
    for path in SOURCES:
        with open(path) as f:
            found += bulk_copies(f.read())
    assert len(found) >= 4
