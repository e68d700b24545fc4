"""The partition of ragged work over a grid, as the kernels' header has it: a host program made from seg_plan.cuh walks
lines of units, and the pieces, owners and slots are checked here.  Needs nvcc but no GPU."""
import subprocess

import numpy as np
import pytest

from gqa_split_kv_gb300 import build as build_mod

PROGRAM = r"""
#include <cstdio>
#include "seg_plan.cuh"
// lines: "d a b" -> a / b; "s W ctas c" -> used, start; "o W ctas x" -> owner; "t len cap base" -> tiles
int main() {
  char what;
  long long a, b, c;
  while (std::scanf(" %c", &what) == 1) {
    if (what == 'd' && std::scanf("%lld %lld", &a, &b) == 2) std::printf("%lld\n", da::seg_div(a, b));
    if (what == 's' && std::scanf("%lld %lld %lld", &a, &b, &c) == 3) {
      const int used = da::seg_used(a, (int)b);
      std::printf("%lld\n", da::seg_start(a, used, (int)c));
    }
    if (what == 'o' && std::scanf("%lld %lld %lld", &a, &b, &c) == 3)
      std::printf("%d\n", da::seg_owner(a, da::seg_used(a, (int)b), c));
    if (what == 't' && std::scanf("%lld %lld %lld", &a, &b, &c) == 3)
      std::printf("%d\n", da::seg_tiles((int)a, (int)b, (int)c));
  }
}
"""


@pytest.fixture(scope="module")
def ask(tmp_path_factory):
    """ask([(what, numbers ...), ...]) -> the program's answers."""
    folder = tmp_path_factory.mktemp("plan")
    source, out = str(folder / "plan.cu"), str(folder / "plan")
    with open(source, "w") as f:
        f.write(PROGRAM)
    made = subprocess.run([build_mod.nvcc_path(), "-std=c++17", "-gencode", "arch=compute_103a,code=sm_103a", "-I",
                           build_mod.CSRC, "-o", out, source], capture_output=True, text=True)
    assert made.returncode == 0, made.stderr

    def run(questions):
        text = "\n".join(" ".join(map(str, q)) for q in questions)
        got = subprocess.run([out], input=text, capture_output=True, text=True, check=True)
        return [int(x) for x in got.stdout.split()]
    return run


def test_division_on_both_sides_of_32_bits(ask):
    edge = 2 ** 32
    pairs = [(a, b) for a in (0, 1, edge - 1, edge, edge + 1, 2 ** 50 + 12345, 608 * 2 ** 40)
             for b in (1, 3, 608, edge - 1, edge, edge + 5)]
    assert ask([("d", a, b) for a, b in pairs]) == [a // b for a, b in pairs]


def test_tiles(ask):
    cases = [(0, 100, 0), (-5, 100, 0), (64, 100, 0), (65, 100, 0), (500, 100, 0), (100, 100, 96), (96, 100, 96),
             (97, 1000, 96), (2 ** 31 - 1, 2 ** 31 - 1025, 0)]
    want = [max(-(-(min(n, cap) - base) // 64), 0) if min(n, cap) > base else 0 for n, cap, base in cases]
    assert ask([("t", *c) for c in cases]) == want


@pytest.mark.parametrize("seed", range(10))
def test_pieces_slots_and_owners(ask, seed):
    """Every tile lies in one CTA's range, ranges differ by a tile at most, the owners of a unit's first and last tile are
    the CTAs of its first and last piece, and no two pieces share a slot unit + CTA."""
    rng = np.random.default_rng(seed)
    tiles = rng.integers(0, 9, rng.integers(1, 60)) * rng.integers(0, 2) + rng.integers(0, 3)
    if seed >= 6:  # lines longer than 2^32 tiles
        tiles = rng.integers(0, 2 ** 33, 20)
    W, ctas = int(tiles.sum()), int(rng.integers(1, 620))
    if W == 0:
        return
    used = min(W, ctas)
    starts = ask([("s", W, ctas, c) for c in range(used + 1)])
    assert starts[0] == 0 and starts[-1] == W
    sizes = np.diff(starts)
    assert sizes.min() >= 1 and sizes.max() - sizes.min() <= 1
    ends = np.cumsum(tiles)
    firsts = [int(e - n) for e, n in zip(ends, tiles)]
    units = [u for u, n in enumerate(tiles) if n]
    owners = ask([("o", W, ctas, x) for u in units for x in (firsts[u], int(ends[u]) - 1)])
    slots = set()
    for k, u in enumerate(units):
        c0, c1 = owners[2 * k], owners[2 * k + 1]
        assert starts[c0] <= firsts[u] < starts[c0 + 1] and starts[c1] < ends[u] <= starts[c1 + 1]
        for c in range(c0, c1 + 1):
            assert u + c not in slots and u + c < len(tiles) + ctas
            slots.add(u + c)
