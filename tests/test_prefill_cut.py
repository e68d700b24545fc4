"""How a latent prefill cuts a query block's keys, compiled for the host."""
import ctypes
import os
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "gqa_split_kv_gb300", "csrc")


@pytest.fixture(scope="module")
def cut(tmp_path_factory):
    d = tmp_path_factory.mktemp("cut")
    src, out = d / "cut.cpp", d / "cut.so"
    src.write_text('#define __host__\n#define __device__\n#include "prefill_cut.cuh"\nextern "C" int block_parts(int t, int p) '
                   '{ return da::prefill_block_parts(t, p); }\nextern "C" int part_begin(int t, int i, int n) '
                   '{ return da::prefill_part_begin(t, i, n); }\nextern "C" int group(int longest, int D, long long units) '
                   '{ return da::prefill_group(longest, D, units); }\n')
    subprocess.run([os.environ.get("CXX", "g++"), "-std=c++17", "-shared", "-fPIC", "-I" + CSRC, str(src), "-o", str(out)],
                   check=True)
    lib = ctypes.CDLL(str(out))
    lib.group.argtypes = [ctypes.c_int, ctypes.c_int, ctypes.c_longlong]
    return lib


def test_never_more_parts_than_the_launch_has(cut):
    """One CTA a block is one part at any length: there are no partials to write then."""
    for tiles in (0, 1, 4, 5, 21, 1000, 0x7fffffff // 256, 0x7fffffff // 256 + 1, (2 ** 31 - 1) // 128 + 1, 2 ** 31 - 1):
        assert cut.block_parts(tiles, 1) == cut.block_parts(tiles, 0) == 1
        for parts in (2, 19, 152):
            assert 1 <= cut.block_parts(tiles, parts) <= parts


def test_equal_parts_that_cover_the_block(cut):
    for parts in (2, 6, 19, 152):
        for tiles in (1, 3, 4, 5, 8, 9, 24, 25, 100, 1024):
            n = cut.block_parts(tiles, parts)
            ends = [cut.part_begin(tiles, i, n) for i in range(n + 1)]
            size = [b - a for a, b in zip(ends, ends[1:])]
            assert ends[0] == 0 and ends[-1] == tiles and max(size) - min(size) <= 1
            assert n == min(parts, -(-tiles // 4)) and min(size) >= 1
    assert cut.block_parts(24, 19) == 6 and cut.block_parts(1024, 19) == 19


def test_launch_groups(cut):
    g = cut.group
    assert g(4096, 128, 32) == 32 and g(131072, 128, 32) == 1 and g(8192, 128, 32) == 24
    for longest in (0, 1, 128, 3000, 2 ** 31 - 1):
        for D in (64, 128):
            for units in (1, 7, 1 << 20):
                n = g(longest, D, units)
                assert 1 <= n <= units and (n == 1 or n * 4 * D * max(longest, 1) <= 96 << 20)
