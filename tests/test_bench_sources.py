"""The captured DRAM bytes are tied to every source that their kernels and launches are built from."""
import os
import re
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)
import bench  # noqa: E402

CSRC = os.path.join(ROOT, "gqa_split_kv_gb300", "csrc")


@pytest.mark.parametrize("kind", sorted(bench.KERNEL_SOURCES))
def test_no_included_source_is_left_out(kind):
    files = bench.KERNEL_SOURCES[kind]
    for f in files:
        for g in re.findall(r'#include "([^"/]+)"', open(os.path.join(CSRC, f)).read()):
            # the decode unit also holds the prefill's host side, which has a list of its own
            assert g in files or (kind, g) == ("decode", "prefill_host.cuh"), (f, g)


def test_the_prefill_list_names_what_its_kernels_use():
    assert {"device_error.cuh", "host_util.cuh"} <= set(bench.KERNEL_SOURCES["prefill"])
