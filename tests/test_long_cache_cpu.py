"""Attention over long caches without a GPU: the oracle against its definitions, what the entry points refuse before
any launch, and the partition of ragged work."""
import itertools

import numpy as np
import pytest

from gqa_split_kv_gb300 import build as build_mod
from oracle import long_cache as ol

A = 0x10000  # a fake aligned address: never dereferenced by rejected calls
BIG = 1 << 40
F = 0.125


@pytest.fixture(scope="module")
def clib():
    build_mod.build()
    from gqa_split_kv_gb300 import binding
    return binding.load()


# ---------------------------------------------------------------- oracle

def test_attend_is_a_softmax_over_what_is_seen():
    rng = np.random.default_rng(0)
    q, k, v = rng.standard_normal((3, 4, 8)), rng.standard_normal((5, 2, 8)), rng.standard_normal((5, 2, 8))
    out, mass = ol.attend(q, k, v, 0.3)
    for i, hq in itertools.product(range(3), range(4)):
        e = [np.exp(0.3 * q[i, hq] @ k[t, hq // 2]) for t in range(5 - 3 + 1 + i)]
        want = sum(x * v[t, hq // 2] for t, x in enumerate(e)) / sum(e)
        assert np.allclose(out[i, hq], want, atol=1e-13)
        assert (mass[i, hq] >= np.abs(out[i, hq]) - 1e-13).all()
    assert not ol.attend(q, k[:2], v[:2], 0.3)[0][0].any()  # the first token sees nothing
    twice, _ = ol.attend(q[2:], k, v, 0.3, [[[0, 0, 1], [0, 0, 1]]])
    e = [np.exp(0.3 * q[2, 0] @ k[t, 0]) for t in (0, 1)]
    assert np.allclose(twice[0, 0], (2 * e[0] * v[0, 0] + e[1] * v[1, 0]) / (2 * e[0] + e[1]), atol=1e-13)


def test_weights_are_the_sums_of_attend():
    rng = np.random.default_rng(1)
    q, k = rng.standard_normal((2, 4, 8)), rng.standard_normal((6, 2, 8))
    w = ol.weights(q, k, 0.5)
    assert np.allclose(w.sum(1), [4, 4])
    for t in range(6):  # values that are 1 at token t alone
        v = np.zeros((6, 2, 8))
        v[t] = 1
        out, _ = ol.attend(q, k, v, 0.5)
        assert np.allclose(w[:, t], out[..., 0].reshape(2, 2, 2).sum((0, 2)))


def test_select_takes_the_best_of_what_is_not_forced():
    means = np.zeros((1, 6, 2))
    means[0, :, 0] = [1, 5, 3, 5, 2, 9]
    q = np.array([[[1.0, 0.0]]])
    assert ol.select(q, means, 12, 2, 3, 1, 1)[0, 0].tolist() == [0, 1, 5]  # ties: the lower block
    assert ol.select(q, means, 12, 2, 4, 0, 1)[0, 0].tolist() == [1, 2, 3, 5]
    assert ol.select(q, means, 4, 2, 4, 0, 1)[0, 0].tolist() == [0, 1, -1, -1]
    assert ol.select(q, means, 0, 2, 2, 0, 1)[0, 0].tolist() == [-1, -1]


def test_evict_orders_special_numbers():
    w = np.array([9, np.nan, 0.0, -0.0, -np.inf, 2, 2, 1])
    assert ol.evict(w, 8, 0, 0).tolist() == list(range(8))
    assert ol.evict(w, 2, 1, 1).tolist() == [0, 7]
    assert ol.evict(w, 3, 1, 1).tolist() == [0, 5, 7]
    assert ol.evict(w, 5, 1, 1).tolist() == [0, 2, 5, 6, 7]
    assert ol.evict(w, 7, 1, 1).tolist() == [0, 2, 3, 4, 5, 6, 7]


# ---------------------------------------------------------------- the partition

def plan(tiles, ctas):
    """Pieces (unit, cta, tiles) of the line of units, as seg_plan.cuh cuts it."""
    W = int(sum(tiles))
    starts = np.cumsum([0] + list(tiles))
    ctas = min(ctas, W)
    for c in range(ctas):
        x, x1 = W * c // ctas, W * (c + 1) // ctas
        while x < x1:
            u = int(np.searchsorted(starts, x, side="right")) - 1
            end = min(x1, int(starts[u + 1]))
            yield u, c, end - x
            x = end


@pytest.mark.parametrize("seed", range(12))
def test_slots_are_their_pieces_own(seed):
    rng = np.random.default_rng(seed)
    tiles = rng.integers(0, 9, rng.integers(1, 60)) * rng.integers(0, 2, 1) + rng.integers(0, 3)
    ctas = int(rng.integers(1, 70))
    pieces = list(plan(tiles, ctas))
    slots = [u + c for u, c, _ in pieces]
    assert len(set(slots)) == len(slots) and all(s < len(tiles) + ctas for s in slots)
    W, starts = int(sum(tiles)), np.cumsum([0] + list(tiles))
    assert sum(n for _, _, n in pieces) == W
    ctas = min(ctas, W)
    for u, n in enumerate(tiles):  # the owners of a unit's first and last tile bound its pieces: a merge walks them all
        if n:
            first, last = (((int(x) + 1) * ctas - 1) // W for x in (starts[u], starts[u + 1] - 1))
            assert [c for v, c, _ in pieces if v == u] == list(range(first, last + 1))


# ---------------------------------------------------------------- refusals

def prefix_contig(clib, q=A, kp=A + BIG, vp=A + 2 * BIG, k=A + 3 * BIG, v=A + 4 * BIG, lens=None, B=1, n=1, Hq=8, Hkv=2,
                  D=64, P=10, ctx=64, scale=F, ws=A + 5 * BIG, size=BIG, out=A + 6 * BIG):
    return clib.prefix_attn_contig(q, kp, vp, k, v, lens, B, n, Hq, Hkv, D, P, ctx, scale, ws, size, out, None)


def prefix_paged(clib, k=A + BIG, pt=A, P=10, table=A, lens=A, D=64, ps=16, cols=8, pages=9, cap=100, ws=A + 5 * BIG,
                 size=BIG, Hq=8):
    return clib.prefix_attn_paged(A, k, A + 2 * BIG, pt, P, table, lens, 1, 1, Hq, 2, D, ps, cols, pages, cap, F, ws, size,
                                  A + 6 * BIG, None)


def test_prefix_refusals(clib):
    f = lambda **kw: prefix_contig(clib, **kw)  # noqa: E731
    assert f(Hq=7) == f(B=-1) == f(n=-1) == f(P=-1) == f(ctx=-1) == f(Hkv=0) == f(scale=float("nan")) == 1
    assert f(D=32) == f(D=96) == f(Hq=130, Hkv=1) == f(P=2 ** 31 - 1, ctx=2 ** 31 - 1) == 2
    assert f(q=None) == f(out=None) == f(k=None) == f(kp=None) == f(vp=None) == 1
    assert f(q=A + 8) == f(out=A + 2) == f(k=A + BIG * 3 + 4) == f(lens=A + 2) == 1
    assert f(out=A) == f(out=A + 3 * BIG) == f(out=A + BIG) == 1  # overlaps
    assert f(B=0) == f(n=0) == 0
    assert f(B=2 ** 20, n=2 ** 20) == 2
    g = lambda **kw: prefix_paged(clib, **kw)  # noqa: E731
    assert g(pt=None) == g(table=None) == g(lens=None) == g(k=None) == g(ps=0) == g(cols=-1) == g(cap=-1) == g(pages=-1) == 1
    assert g(ps=24) == g(D=48) == 2
    assert clib.prefix_attn_workspace_bytes(4, 1, 8, 2, 128, 152) > 0
    assert clib.prefix_attn_workspace_bytes(4, 1, 8, 2, 100, 152) == -2
    assert clib.prefix_attn_workspace_bytes(4, 1, 8, 3, 128, 152) == -1


def test_sparse_refusals(clib):
    def means(k=A, lens=None, B=1, n=1, H=2, D=64, ctx=128, block=64, blocks=2, out=A + BIG):
        return clib.block_means_contig(k, lens, B, n, H, D, ctx, block, blocks, out, None)
    assert means(block=0) == means(blocks=1) == means(B=-1) == means(k=None) == means(out=A) == means(k=A + 4) == 1
    assert means(D=12) == means(D=2048) == 2
    assert means(B=0) == means(n=0) == means(ctx=0) == 0

    def select(q=A, m=A + BIG, B=1, n=1, Hq=8, Hkv=2, D=64, block=64, blocks=9, pick=4, first=1, recent=1,
               out=A + 2 * BIG):
        return clib.block_select(q, m, None, B, n, Hq, Hkv, D, block, blocks, pick, first, recent, out, None)
    assert select(pick=0) == select(first=-1) == select(recent=0) == select(first=4) == select(block=0) == 1
    assert select(q=None) == select(m=None) == select(out=A) == select(out=A + BIG) == select(q=A + 4) == 1
    assert select(D=32) == select(blocks=8193) == select(Hq=200, Hkv=2) == 2
    assert select(B=0) == 0

    def sparse(q=A, k=A + BIG, v=A + 2 * BIG, blocks=A, B=1, n=1, Hq=8, Hkv=2, D=64, ctx=128, block=64, pick=2, scale=F,
               out=A + 4 * BIG):
        return clib.sparse_attn_contig(q, k, v, blocks, None, B, n, Hq, Hkv, D, ctx, block, pick, scale, out, None)
    assert sparse(pick=0) == sparse(block=0) == sparse(blocks=None) == sparse(blocks=A + 2) == sparse(scale=float("inf")) == 1
    assert sparse(out=A) == sparse(out=A + BIG) == sparse(k=None) == sparse(Hq=9) == sparse(ctx=-1) == 1
    assert sparse(block=24) == sparse(D=80) == sparse(pick=2 ** 26, block=64) == 2


def test_weights_refusals(clib):
    def weights(q=A, k=A + BIG, B=1, n=1, Hq=8, Hkv=2, D=64, ctx=64, scale=F, decay=1.0, prior=None, ws=A + 3 * BIG,
                size=BIG, out=A + 2 * BIG):
        return clib.kv_weights_contig(q, k, None, B, n, Hq, Hkv, D, ctx, scale, decay, prior, ws, size, out, None)
    assert weights(decay=float("nan")) == weights(scale=float("inf")) == weights(k=None) == weights(out=None) == 1
    assert weights(out=A) == weights(prior=A + 2 * BIG + 4) == weights(prior=A + 2) == weights(ctx=-1) == weights(Hq=9) == 1
    assert weights(D=96) == weights(n=257) == 2
    assert weights(B=0) == weights(ctx=0) == 0
    assert clib.kv_weights_int8_contig(A, A + BIG, None, None, 1, 1, 8, 2, 64, 64, F, 1.0, None, A, BIG, A + 2 * BIG, None) == 1
    assert clib.kv_weights_paged(A, A + BIG, A, A, 1, 1, 8, 2, 64, 24, 4, 9, 64, F, 1.0, None, A, BIG, A + 2 * BIG, None) == 2
    assert clib.kv_weights_workspace_bytes(2, 1, 8, 2, 1000, 152) > 0
    assert clib.kv_weights_workspace_bytes(2, 1, 8, 2, -1, 152) == -1


def test_evict_refusals(clib):
    def evict(k=A, v=A + BIG, w=A + 2 * BIG, lens=None, B=1, H=2, D=64, ctx=64, keep=8, first=1, recent=1, ko=None, vo=None,
              wo=None, oc=0, kept=A + 6 * BIG, nl=A + 7 * BIG):
        return clib.kv_evict_contig(k, v, w, lens, B, H, D, ctx, keep, first, recent, ko, vo, wo, oc, kept, nl, None)
    assert evict(keep=0) == evict(first=-1) == evict(recent=-1) == evict(first=5, recent=4) == evict(H=0) == 1
    assert evict(k=None) == evict(w=None) == evict(kept=None) == evict(nl=None) == evict(k=A + 8) == evict(w=A + 2) == 1
    assert evict(v=A) == evict(kept=A) == evict(nl=A + 6 * BIG) == evict(w=A) == evict(lens=A + 6 * BIG) == 1
    assert evict(vo=A + 3 * BIG) == evict(wo=A + 3 * BIG) == evict(ko=A + 3 * BIG) == 1  # some of the outputs
    out = dict(ko=A + 3 * BIG, vo=A + 4 * BIG)
    assert evict(**out, oc=7) == evict(ko=A, vo=A + 4 * BIG, oc=8) == evict(ko=A + 3 * BIG, vo=A + 3 * BIG, oc=8) == 1
    assert evict(D=4) == evict(D=2048) == evict(ctx=2 ** 31 - 1) == 2
    assert evict(B=0) == 0
    assert clib.kv_evict_int8_contig(A, A + BIG, None, None, A + 2 * BIG, None, 1, 2, 64, 64, 8, 1, 1, None, None, None, None,
                                     None, 0, A + 6 * BIG, A + 7 * BIG, None) == 1
    assert clib.kv_evict_paged(A, A + BIG, A + 2 * BIG, None, A, 1, 2, 64, 16, 4, 9, 64, 8, 1, 1, None, None, None, 0,
                               A + 6 * BIG, A + 7 * BIG, None) == 1


def test_sizes_whose_loops_would_pass_32_bits(clib):
    most = 2 ** 31 - 1
    assert prefix_contig(clib, ctx=most - 600) == prefix_contig(clib, P=most - 600, ctx=0) == 2
    assert clib.kv_weights_contig(A, A + BIG, None, 1, 1, 8, 2, 64, most - 600, F, 1.0, None, A, BIG, A + 2 * BIG, None) == 2
    assert clib.block_select(A, A + BIG, None, 1, 1, 8, 2, 64, 64, 9, most, 1, 1, A + 2 * BIG, None) == 2
    assert clib.sparse_attn_contig(A, A + BIG, A + 2 * BIG, A, None, 1, 1, 8, 2, 64, most - 600, 64, 2, F, A + 4 * BIG, None) == 2
    out = (A + 6 * BIG, A + 7 * BIG, None)
    assert clib.kv_evict_contig(A, A + BIG, A + 2 * BIG, None, 1, 2, 64, 64, most, 1, 1, None, None, None, 0, *out) == 2
    assert clib.kv_evict_contig(A, A + BIG, A + 2 * BIG, None, 1, 2, 64, 64, 8, 1, 1, A + 3 * BIG, A + 4 * BIG, None, most,
                                *out) == 2
