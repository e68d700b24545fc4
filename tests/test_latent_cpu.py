"""Latent attention without a GPU: the oracle's pins and what the entry points refuse."""
import ctypes
import math

import numpy as np
import pytest

from oracle import latent_attention as ol
from gqa_split_kv_gb300 import build as build_mod

A = 0x10000  # aligned addresses, far apart, that refused calls never read
K, V, PE, WS, OUT = (A + (i << 44) for i in range(1, 6))


@pytest.fixture(scope="module")
def clib():
    build_mod.build()
    from gqa_split_kv_gb300 import binding
    return binding.load()


# ---------------------------------------------------------------- the oracle

def test_absorbed_is_attention_with_the_cache_as_keys_and_values():
    rng = np.random.default_rng(0)
    q, c = rng.standard_normal((1, 3, 10)), rng.standard_normal((7, 10))
    got = ol.absorbed(q, c, 6, 0.3)
    for h in range(3):
        s = [0.3 * sum(float(a) * float(b) for a, b in zip(q[0, h], row)) for row in c]
        w = [math.exp(x) for x in s]
        ref = [sum(wi * row[r] for wi, row in zip(w, c)) / sum(w) for r in range(6)]
        assert np.allclose(got[0, h], ref, rtol=1e-13)


def test_one_token_and_no_token():
    c = np.arange(8.0)[None]
    q = np.ones((3, 2, 8))
    out = ol.absorbed(q, c, 5, 1.0)  # of 3 queries the last alone sees the one token
    assert np.array_equal(out[2], np.tile(c[:, :5], (2, 1))) and not out[:2].any()


def test_expanded_equals_absorbed():
    rng = np.random.default_rng(1)
    L, H, D, R, P = 9, 2, 3, 4, 2
    c = rng.standard_normal((L, R + P))
    uk, uv = rng.standard_normal((2, H, D, R))
    qn, qr = rng.standard_normal((4, H, D)), rng.standard_normal((4, H, P))
    a = ol.absorbed(np.concatenate([np.einsum("ihd,hdr->ihr", qn, uk), qr], -1), c, R, 0.3)
    e = ol.expanded(np.concatenate([qn, qr], -1), np.einsum("tr,hdr->thd", c[:, :R], uk), c[:, R:],
                    np.einsum("tr,hdr->thd", c[:, :R], uv), 0.3)
    assert np.allclose(np.einsum("ihr,hdr->ihd", a, uv), e, atol=1e-13)


def test_causal_and_pages():
    rng = np.random.default_rng(2)
    c, q = rng.standard_normal((12, 6)), rng.standard_normal((3, 2, 6))
    out = ol.absorbed(q, c, 4, 0.5)
    for i in range(3):
        assert np.allclose(out[i], ol.absorbed(q[i:i + 1], c[:10 + i], 4, 0.5)[0], rtol=1e-13)
    pool = np.zeros((5, 4, 6))
    table = np.array([3, 0, 4])
    for t in range(12):
        pool[table[t // 4], t % 4] = c[t]
    assert np.array_equal(ol.gather_rows(pool, table, 12, 4), c)


# ---------------------------------------------------------------- refusals

def attn(clib, paged=False, q=A, cache=K, table=A, lens=A, B=2, n=1, H=16, R=512, ctx=64, ps=16, maxp=4, npages=8,
         maxlen=64, scale=0.1, ws=WS, size=1 << 40, out=OUT):
    f = ctypes.c_float(scale)
    if paged:
        return clib.latent_attn_paged(q, cache, table, lens, B, n, H, R, ps, maxp, npages, maxlen, f, ws, size, out, None)
    return clib.latent_attn_contig(q, cache, lens, B, n, H, R, ctx, f, ws, size, out, None)


@pytest.mark.parametrize("kw,want", [
    (dict(B=-1), 1), (dict(n=0), 1), (dict(n=17), 1), (dict(H=0), 1), (dict(H=257), 2), (dict(R=64), 2),
    (dict(R=384), 2), (dict(ctx=-1), 1), (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1),
    (dict(q=None), 1), (dict(out=None), 1), (dict(q=A + 8), 1), (dict(out=OUT + 2), 1), (dict(cache=None), 1),
    (dict(cache=K + 8), 1), (dict(lens=A + 2), 1), (dict(B=1 << 20), 2), (dict(B=0), 0),
    (dict(paged=True, ps=0), 1), (dict(paged=True, ps=24), 2), (dict(paged=True, ps=8), 2),
    (dict(paged=True, maxp=-1), 1), (dict(paged=True, npages=-1), 1), (dict(paged=True, maxlen=-1), 1),
    (dict(paged=True, table=None), 1), (dict(paged=True, lens=None), 1), (dict(paged=True, table=A + 2), 1),
    (dict(paged=True, maxp=1 << 30, ps=64, maxlen=2 ** 31 - 1, B=0), 0),
])
def test_attention_refusals(clib, kw, want):
    assert attn(clib, **kw) == want


def test_workspace_and_batch_queries(clib):
    size = clib.latent_workspace_bytes
    assert size(1, 1, 64, 512, 152) == 2 * 152 * 64 * (512 * 4 + 8) + (152 + 1) * 16
    assert size(4, 2, 64, 512, 152) == 2 * 152 * 64 * (512 * 4 + 8) + (152 + 4 * 2) * 16
    assert size(1, 1, 5, 128, 152) == 2 * 152 * 16 * (128 * 4 + 8) + (152 + 1) * 16
    assert size(1, 1, 64, 500, 152) == -2 and size(1, 0, 64, 512, 152) == -1
    assert clib.latent_max_batch(1, 64, 512) >= 8192 and clib.latent_max_batch(1, 1, 100) == -2
    assert clib.latent_max_batch(0, 1, 128) == -1


def prefill(clib, q=A, k=K, pe=PE, v=V, lens=A, B=2, n=4, H=4, D=128, ctx=64, ts=512, hs=128, ps=64, scale=0.1, out=OUT,
            ws=None, size=0):
    return clib.latent_prefill_contig(q, k, pe, v, lens, B, n, H, D, ctx, ts, hs, ps, ctypes.c_float(scale), ws, size, out,
                                      None)


@pytest.mark.parametrize("kw,want", [
    (dict(B=-1), 1), (dict(n=-1), 1), (dict(H=0), 1), (dict(D=96), 2), (dict(D=256), 2), (dict(ctx=-1), 1),
    (dict(scale=float("nan")), 1), (dict(q=None), 1), (dict(k=None), 1), (dict(pe=None), 1), (dict(v=None), 1),
    (dict(out=None), 1), (dict(q=A + 8), 1), (dict(k=K + 8), 1), (dict(pe=PE + 4), 1), (dict(v=V + 2), 1),
    (dict(out=OUT + 8), 1), (dict(lens=A + 1), 1), (dict(ws=WS + 8), 1), (dict(ts=1 << 41), 1),
    (dict(out=A), 1), (dict(out=V + 16), 1), (dict(out=PE), 1), (dict(ws=K, size=64), 1), (dict(ws=OUT, size=64), 1), (dict(hs=64), 1), (dict(hs=132, ts=1024), 1), (dict(ts=500), 1),
    (dict(ts=516), 1), (dict(ps=32), 1), (dict(ps=68), 1), (dict(B=1 << 20, n=1 << 20), 2), (dict(B=0), 0), (dict(n=0), 0),
])
def test_prefill_refusals(clib, kw, want):
    assert prefill(clib, **kw) == want


def test_prefill_workspace(clib):
    size = clib.latent_prefill_workspace_bytes
    assert size(1, 4096, 64, 128, 4096, 152) == 0          # 1024 blocks fill the card
    assert size(4, 500, 16, 128, 3000, 152) == 0           # 128 blocks: two parts each would not run at once
    assert size(1, 256, 16, 128, 512, 152) == 0            # 4 tiles are one part
    # 32 blocks: 4 parts each run at once, of 24 tiles
    assert size(4, 200, 8, 128, 3000, 152) == 32 * 4 * 256 * (128 + 2) * 4
    assert size(1, 1, 1, 64, 100000, 152) == 152 * 256 * (64 + 2) * 4  # one block: the whole card
    assert size(1, 1, 1, 64, 1000, 152) == 2 * 256 * (64 + 2) * 4      # 8 tiles: two parts of 4
    assert size(0, 5, 4, 128, 3000, 152) == 0 and size(1, 5, 4, 96, 3000, 152) == -2 and size(-1, 5, 4, 64, 1, 152) == -1


def test_binding_refuses_mismatched_tensors():
    torch = pytest.importorskip("torch")
    from gqa_split_kv_gb300 import binding
    z = lambda *s, t=torch.bfloat16: torch.zeros(s, dtype=t)  # noqa: E731
    i32 = torch.int32
    for q, cache, lens in ((z(2, 1, 4, 192), z(3, 8, 192), None), (z(2, 1, 4, 192), z(2, 8, 200), None),
                           (z(2, 4, 192), z(2, 8, 192), None), (z(2, 1, 4, 192), z(2, 8, 1, 192), None),
                           (z(2, 1, 4, 192, t=torch.float16), z(2, 8, 192), None),
                           (z(2, 1, 4, 192), z(2, 8, 192), z(2, t=torch.int64)),
                           (z(2, 1, 4, 192), z(2, 8, 192), None)):  # last: on the CPU
        with pytest.raises(ValueError):
            binding.latent_attn_contig(q, cache, lens, scale=1.0)
    with pytest.raises(ValueError):
        binding.latent_attn_paged(z(2, 1, 4, 192), z(5, 16, 192), z(3, 2, t=i32), z(2, t=i32), 32, scale=1.0)
    with pytest.raises(ValueError):
        binding.latent_attn_paged(z(2, 1, 4, 192), z(5, 16, 192), z(2, 2, t=i32), None, 32, scale=1.0)
    q, k, pe = z(2, 3, 4, 128), z(2, 8, 4, 64), z(2, 8, 64)
    for a in ((q, z(2, 8, 4, 32), pe, k), (q, k, z(2, 7, 64), k), (q, k, pe, z(2, 8, 3, 64)), (q[0], k, pe, k),
              (q, k, pe, z(2, 8, 4, 128)[..., :64]), (q, z(2, 4, 8, 64).transpose(1, 2), pe, k), (q, k, pe, k)):
        with pytest.raises(ValueError):
            binding.latent_prefill_contig(*a, scale=1.0)
    with pytest.raises(binding.DecodeAttnError):
        binding.latent_max_batch(4, 100)


def test_extents_past_64_bits_are_refused(clib):
    most, far, ctx = 2 ** 31 - 1, 1 << 40, 2 ** 31 - 512
    assert prefill(clib, B=1 << 20, ctx=ctx, ts=far) == 1 and prefill(clib, B=1 << 20, ctx=ctx, ps=far) == 1
    assert prefill(clib, H=1 << 20, n=1, hs=far, ts=far) == 1
    # pools whose bytes pass 2^64 still share them with whatever lies behind their start
    big = dict(paged=True, B=1, ps=1 << 30, npages=most, maxp=1, maxlen=64)
    assert attn(clib, **big, out=K + (1 << 43)) == 1 and attn(clib, **big, ws=K + (1 << 43)) == 1


@pytest.mark.parametrize("ctx", [2 ** 31 - 1, 2 ** 31 - 128])
def test_prefill_refuses_lengths_whose_last_tile_passes_32_bits(clib, ctx):
    """Keys, values and shared parts in one tensor of 64 columns would fit the card at 2^31 tokens."""
    assert prefill(clib, B=1, H=1, D=64, ctx=ctx, ts=64, hs=64, ps=64, k=K, v=K, pe=K, out=A + (1 << 30)) == 2
