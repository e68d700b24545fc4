"""Kernels launched as programmatic dependents start while the kernel before them may still be writing their
inputs.  The read-only load path (__ldg, ld.global.nc) is for memory that nothing writes while the grid lives, so no
source that such a kernel is built from may use it.  Reads the sources; needs no GPU."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "gqa_split_kv_gb300", "csrc")


def code(name):
    text = open(os.path.join(CSRC, name)).read()
    return re.sub(r"//[^\n]*|/\*.*?\*/", "", text, flags=re.S)


def sources_of(unit):
    """The unit and every file of this folder that it includes."""
    found, todo = set(), [unit]
    while todo:
        name = todo.pop()
        if name not in found:
            found.add(name)
            todo += [f for f in re.findall(r'#include "([^"]+)"', code(name)) if os.path.exists(os.path.join(CSRC, f))]
    return sorted(found)


UNITS = [f for f in sorted(os.listdir(CSRC)) if f.endswith(".cu") and re.search(r"\blaunch_dependent\(", code(f))]


def test_the_dependent_units_are_found():
    assert {"cache_ops.cu", "latent_attn.cu"} <= set(UNITS)


@pytest.mark.parametrize("name", sorted({f for u in UNITS for f in sources_of(u)}))
def test_no_read_only_loads(name):
    assert not re.findall(r"__ldg\b|ld\.global\S*\.nc\b", code(name)), name
