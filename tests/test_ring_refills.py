"""A warp that copies into its own ring of keys with cp.async overwrites what its lanes have read with ordinary loads, so
a warp barrier stands between the two: lanes may run apart.  Reads the sources; needs no GPU."""
import re

import pytest

from test_dependent_loads import code


def loop_of(name, head):
    text = re.sub(r"\s+", " ", code(name))
    return text[text.index(head):]


@pytest.mark.parametrize("name,head,refill", [
    ("weights_kernel.cuh", "for (long long x = x0; x < x1; ++x) {", "ring.issue(stage);"),
    ("seg_kernel.cuh", "for (long long x = x0; x < x1; ++x) {", "if (!join) issue();"),
])
def test_a_barrier_stands_before_a_refill(name, head, refill):
    loop = loop_of(name, head)
    before = loop[:loop.index(refill)].rstrip()
    assert before.endswith("__syncwarp();"), (name, before[-120:])


def test_a_barrier_stands_behind_the_last_read_of_a_tile():
    """seg_kernel's second refill, at a tile's end: behind the products with the values, or the join's barriers."""
    loop = loop_of("seg_kernel.cuh", "for (long long x = x0; x < x1; ++x) {")
    values = loop.rindex("ldsm_x4_t(")
    assert "__syncwarp(); if (join) {" in loop[values:loop.index("issue(); ++j;")]
