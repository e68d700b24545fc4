"""Rotary positions, cache writes and cache reads without a GPU: the oracle's pins, the
frequency tables and what the entry points refuse."""
import ctypes
import math

import numpy as np
import pytest

from oracle import cache_ops as oc
from gqa_split_kv_gb300 import build as build_mod

A = 0x10000  # aligned addresses, far apart, that refused calls never read
K, V, SK, SV = (A + (i << 40) for i in range(1, 5))
NAN = float("nan")


@pytest.fixture(scope="module")
def clib():
    build_mod.build()
    from gqa_split_kv_gb300 import binding
    return binding.load()


# ---------------------------------------------------------------- the oracle

@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_is_the_textbook_one(interleaved):
    x = np.array([[1.0, 2.0, 3.0, 4.0, 9.0]])
    w = np.array([0.5, 0.25])
    y = oc.rotate(x, np.array(3), w, 0, interleaved, 2.0)
    pairs = [(0, 1), (2, 3)] if interleaved else [(0, 2), (1, 3)]
    for (a, b), f in zip(pairs, w):
        c, s = math.cos(3 * f), math.sin(3 * f)
        assert y[0, a] == pytest.approx(2 * (x[0, a] * c - x[0, b] * s), rel=1e-14)
        assert y[0, b] == pytest.approx(2 * (x[0, a] * s + x[0, b] * c), rel=1e-14)
    assert y[0, 4] == 9.0


def test_scores_of_rotated_heads_depend_on_the_distance_alone():
    rng = np.random.default_rng(0)
    w = 10000.0 ** (-np.arange(8) / 8)
    q, k = rng.standard_normal((2, 1, 16))
    def dot(p, t):
        return float((oc.rotate(q, np.array(p), w) * oc.rotate(k, np.array(t), w)).sum())
    assert dot(105, 100) == pytest.approx(dot(9, 4), rel=1e-11)


def test_gradient_is_the_transpose():
    rng = np.random.default_rng(1)
    w = rng.random(4)
    x, g = rng.standard_normal((2, 3, 2, 11))
    p = np.array([0, 7, -3])
    for il in (False, True):
        y = oc.rotate(x, p, w, 2, il, 1.3)
        gx = oc.rotate(g, p, w, 2, il, 1.3, backward=True)
        # <g, y(x)> is bilinear: the rest of the head has the identity
        assert (g * y).sum() == pytest.approx((gx * x).sum(), rel=1e-12)


def test_quantize():
    x = np.array([[0.0, 0.0], [1.0, -127.0], [0.5, 1.0], [np.inf, 1.0], [np.nan, 2.0], [1e-44, 0.0]], np.float32)
    q, s = oc.quantize(x)
    assert q[:3].tolist() == [[0, 0], [1, -127], [64, 127]]  # 63.5 to even
    assert s[0] == 1 and s[1] == 1 and np.isnan(s[3]) and np.isnan(s[4]) and not q[3:5].any()
    assert s[5] == np.finfo(np.float32).tiny and not q[5].any()


# ---------------------------------------------------------------- rope_inv_freq

def table(clib, rot, base=10000.0, scaling=0, factor=1.0, ctx=4096.0, low=1.0, high=32.0):
    w = (ctypes.c_double * max(rot // 2, 1))()
    st = clib.rope_inv_freq(w, rot, base, scaling, factor, ctx, low, high)
    return st, np.array(w)


def test_frequencies(clib):
    st, w = table(clib, 64)
    assert st == 0 and np.allclose(w, 10000.0 ** (-np.arange(32) / 32), rtol=1e-15)
    assert np.allclose(table(clib, 64, scaling=1, factor=4.0)[1], w / 4, rtol=1e-15)
    b = table(clib, 64, scaling=2, factor=4.0)[1]  # the fastest pair kept, the slowest stretched by the factor
    assert b[0] == 1 and b[-1] == pytest.approx(w[-1] / 4, rel=1e-13)
    p = table(clib, 64, scaling=3, factor=4.0)[1]
    turns = 4096 * w / (2 * math.pi)
    assert np.array_equal(p[turns > 32], w[turns > 32]) and np.allclose(p[turns < 1], w[turns < 1] / 4, rtol=1e-15)
    mid = (turns > 1) & (turns < 32)
    assert mid.any() and np.all((p[mid] < w[mid]) & (p[mid] > w[mid] / 4))
    assert table(clib, 2)[1][0] == 1


@pytest.mark.parametrize("kw,want", [
    (dict(rot=0), 1), (dict(rot=7), 1), (dict(rot=-2), 1), (dict(rot=8, base=1.0), 1), (dict(rot=8, base=NAN), 1),
    (dict(rot=8, base=float("inf")), 1), (dict(rot=8, scaling=4), 2), (dict(rot=8, scaling=-1), 2),
    (dict(rot=8, scaling=1, factor=0.5), 1), (dict(rot=8, scaling=1, factor=NAN), 1),
    (dict(rot=2, scaling=2, factor=2.0), 1), (dict(rot=8, scaling=3, factor=2.0, ctx=0.0), 1),
    (dict(rot=8, scaling=3, factor=2.0, low=5.0, high=5.0), 1), (dict(rot=8, scaling=3, factor=2.0, low=-1.0), 1),
])
def test_frequency_refusals(clib, kw, want):
    assert table(clib, **kw)[0] == want


# ---------------------------------------------------------------- refusals

def rope(clib, x=A, out=A + 0x100000, pos=A, w=A, T=4, H=2, D=64, off=0, rot=64, il=0, mag=1.0, dtype=0, xt=128,
         xh=64, ot=128, oh=64):
    return clib.rope_apply(x, out, pos, w, T, H, D, off, rot, il, mag, 0, dtype, xt, xh, ot, oh, None)


@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), 1), (dict(H=0), 1), (dict(D=0), 1), (dict(dtype=3), 2), (dict(dtype=-1), 2), (dict(w=None), 1),
    (dict(rot=63), 1), (dict(rot=0), 1), (dict(off=-2), 1), (dict(off=2), 1), (dict(il=2), 1), (dict(mag=NAN), 1),
    (dict(D=5000, rot=4096, xt=10000, xh=5000, ot=10000, oh=5000), 2),
    (dict(x=None), 1), (dict(out=None), 1), (dict(pos=None), 1), (dict(x=A + 1), 1), (dict(out=A + 0x100001), 1),
    (dict(pos=A + 2), 1), (dict(w=A + 4), 1), (dict(dtype=2, x=A + 2), 1), (dict(xt=-1), 1),
    (dict(oh=32), 1), (dict(ot=64), 1), (dict(ot=0), 1),     # rows of out share elements
    (dict(out=A, ot=256), 1),                                # in place with other strides
    (dict(out=A + 16), 1), (dict(out=A - 16), 1),            # overlaps
    (dict(T=0), 0),
])
def test_rope_refusals(clib, kw, want):
    assert rope(clib, **kw) == want


def write(clib, paged=True, int8=True, k_new=A, v_new=A, ks=256, vs=256, table=A, lens=A, B=2, n=1, H=2, D=64, ps=16,
          maxp=4, npages=8, maxlen=64, w=None, off=0, rot=0, il=0, mag=1.0, k=K, v=V, sk=SK, sv=SV):
    where = (ps, maxp, npages, maxlen) if paged else (maxlen,)
    fn = getattr(clib, "kv_write" + ("_int8" if int8 else "") + ("_paged" if paged else "_contig"))
    return fn(k_new, v_new, ks, vs, *((table,) if paged else ()), lens, B, n, H, D, *where, w, off, rot, il, mag, k, v,
              *((sk, sv) if int8 else ()), None)


@pytest.mark.parametrize("kw,want", [
    (dict(B=-1), 1), (dict(n=-1), 1), (dict(H=0), 1), (dict(D=0), 1), (dict(D=24), 2), (dict(D=20, int8=False), 2),
    (dict(D=1040), 2), (dict(H=2000), 2), (dict(ps=0), 1), (dict(maxp=-1), 1), (dict(npages=-1), 1),
    (dict(maxlen=-1), 1), (dict(maxlen=-1, paged=False), 1), (dict(k_new=None), 1), (dict(k_new=A + 8), 1),
    (dict(v_new=None), 1), (dict(v=None), 1), (dict(k=None), 1), (dict(k=K + 8), 1), (dict(sk=None), 1),
    (dict(sv=None), 1), (dict(table=None), 1), (dict(lens=None), 1), (dict(ks=100), 1), (dict(ks=260), 1),
    (dict(vs=64), 1), (dict(w=A, rot=64, off=8), 1), (dict(w=A, rot=24), 2), (dict(w=A, rot=32, off=4), 2),
    (dict(w=A + 4, rot=32), 1), (dict(w=A, rot=0), 1), (dict(w=A, rot=32, il=5), 1), (dict(w=A, rot=32, mag=NAN), 1),
    (dict(B=70000, n=70000), 2), (dict(maxp=1 << 30, ps=64, maxlen=2**31 - 1), None),
    (dict(B=0), 0), (dict(n=0), 0), (dict(ks=1 << 41), 1),
    (dict(k=A), 1), (dict(v=A + 64), 1), (dict(sk=A), 1), (dict(v_new=SV + 16), 1),  # new tokens in the cache
    (dict(v=K), 1), (dict(sv=V), 1), (dict(sk=SV + 4), 1),                          # the cache's tensors share bytes
])
def test_write_refusals(clib, kw, want):
    if want is None:  # a long cap is the smaller of the two: fine up to 2^31 - 1 (refused here for its null table)
        assert write(clib, **kw, table=None) == 1
    else:
        assert write(clib, **kw) == want


def read(clib, paged=True, int8=True, k=K, v=V, sk=SK, sv=SV, table=A, starts=None, lens=A, B=2, n=4, H=2, D=64, ps=16,
         maxp=4, npages=8, maxlen=64, ko=A, vo=A + (1 << 30)):
    where = (ps, maxp, npages, maxlen) if paged else (maxlen,)
    fn = getattr(clib, "kv_read" + ("_int8" if int8 else "") + ("_paged" if paged else "_contig"))
    return fn(k, v, *((sk, sv) if int8 else ()), *((table,) if paged else ()), starts, lens, B, n, H, D, *where, ko, vo,
              None)


@pytest.mark.parametrize("kw,want", [
    (dict(B=-1), 1), (dict(n=-1), 1), (dict(D=24), 2), (dict(D=20, int8=False), 2), (dict(k=None), 1),
    (dict(ko=None), 1), (dict(vo=None), 1), (dict(v=None), 1), (dict(ko=A + 8), 1), (dict(vo=A + 4), 1),
    (dict(sk=None), 1), (dict(sv=None), 1), (dict(table=None), 1), (dict(lens=None), 1), (dict(starts=A + 2), 1),
    (dict(ps=-16), 1), (dict(npages=-1), 1), (dict(maxlen=-1), 1), (dict(paged=False, maxlen=-1), 1),
    (dict(B=0), 0), (dict(n=0), 0), (dict(ko=K), 1), (dict(vo=SV + 16), 1), (dict(vo=A), 1),  # outputs in the cache
    (dict(npages=0, k=None, v=None, sk=None, sv=None), 0), (dict(maxlen=0, k=None, v=None, sk=None, sv=None), 0),
])
def test_read_refusals(clib, kw, want):
    assert read(clib, **kw) == want


def test_binding_refuses_mismatched_tensors():
    torch = pytest.importorskip("torch")
    from gqa_split_kv_gb300 import binding
    bf, i8, f32, i32 = torch.bfloat16, torch.int8, torch.float32, torch.int32
    z = lambda *s, t=bf: torch.zeros(s, dtype=t)  # noqa: E731
    new, pool, scale, tab, lens = z(2, 3, 4, 32), z(8, 16, 4, 32, t=i8), z(8, 4, 16, t=f32), z(2, 5, t=i32), z(2, t=i32)

    def w(k_new=new, v_new=new, k=pool, v=pool, ks=scale, vs=scale, table=tab, L=lens):
        return binding.kv_write_int8_paged(k_new, v_new, k, v, ks, vs, table, L, 80)

    for kw in (dict(k_new=z(2, 3, 4, 16)), dict(v_new=None), dict(v=None), dict(k=z(8, 16, 4, 32)), dict(ks=None),
               dict(vs=None), dict(ks=z(8, 16, 4, t=f32)), dict(vs=z(7, 4, 16, t=f32)), dict(table=z(3, 5, t=i32)),
               dict(table=z(2, 5, t=torch.int64)), dict(L=z(3, t=i32)), dict(L=None), dict(k_new=z(2, 3, 4, 32, t=f32)),
               dict(v=z(8, 16, 2, 32, t=i8)), dict(k_new=z(2, 4, 3, 32).transpose(1, 2)), dict()):  # last: CPU tensors
        with pytest.raises(ValueError):
            w(**kw)
    for kw in (dict(x=z(4, 2, 8, t=torch.float64)), dict(x=z(4, 8)), dict(p=z(4, t=torch.int64)), dict(p=z(3, t=i32)),
               dict(f=z(4)), dict(out=z(4, 2, 9)), dict(x=z(4, 2, 16)[..., ::2])):
        with pytest.raises(ValueError):
            args = dict(dict(x=z(4, 2, 8), p=z(4, t=i32), f=z(4, t=torch.float64), out=z(4, 2, 8)), **kw)
            binding.rope_apply(args["x"], args["p"], args["f"], out=args["out"])
    with pytest.raises(ValueError):
        binding.rope_inv_freq(8, scaling="sideways", device="cpu")
    with pytest.raises(binding.DecodeAttnError):
        binding.rope_inv_freq(7, device="cpu")


@pytest.mark.parametrize("name", ["kv_read_paged", "kv_read_int8_contig", "kv_read_int8_paged"])
def test_filled_reads_refuse_what_reads_refuse(clib, name):
    f, g = getattr(clib, name), getattr(clib, name + "_filled")
    scales = (SK, SV) if "int8" in name else ()
    where = (16, 4, 8, 64) if "paged" in name else (64,)
    table = (A,) if "paged" in name else ()
    for B, n, D, ko, want in ((-1, 4, 64, A, 1), (2, -1, 64, A, 1), (2, 4, 20, A, 2), (2, 4, 64, None, 1),
                              (2, 4, 64, K, 1), (0, 4, 64, A, 0), (2, 0, 64, A, 0)):
        args = (K, V, *scales, *table, None, A, B, n, 2, D, *where, ko, A + (1 << 30), None)
        assert f(*args) == g(*args) == want


def test_outputs_that_autograd_tracks_are_refused():
    torch = pytest.importorskip("torch")
    from gqa_split_kv_gb300 import binding
    x = torch.zeros(4, 2, 8, requires_grad=True)
    pos, w = torch.zeros(4, dtype=torch.int32), torch.zeros(4, dtype=torch.float64)
    for out in (x, x * 1):
        with pytest.raises(ValueError, match="requires a gradient"):
            binding.rope_apply(x.detach(), pos, w, out=out)
    with pytest.raises(ValueError, match="CUDA"):  # under no_grad only the device is wrong here
        with torch.no_grad():
            binding.rope_apply(x, pos, w, out=x)
    k = torch.zeros(1, 4, 1, 8, dtype=torch.bfloat16, requires_grad=True)
    with pytest.raises(ValueError, match="k: it requires a gradient"):
        binding.kv_write_contig(k.detach(), None, k, None)


FAR, MOST = 1 << 40, 2 ** 31 - 1


@pytest.mark.parametrize("kw", [dict(xt=FAR), dict(ot=FAR), dict(xt=FAR, ot=FAR), dict(xt=1 << 33), dict(ot=1 << 33)])
def test_rope_refuses_extents_past_64_bits(clib, kw):
    """2^31 tokens 2^40 elements apart: no such tensor exists, and its size would not fit the overlap checks."""
    assert rope(clib, **{**dict(T=MOST, xt=128, ot=128, out=A + (1 << 45)), **kw}) == 1


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("paged", [False, True])
def test_cache_calls_refuse_extents_past_64_bits(clib, paged, int8):
    far = dict(paged=paged, int8=int8, B=MOST, n=1, maxlen=64)
    assert write(clib, **far, ks=FAR) == 1 and write(clib, **far, vs=1 << 32) == 1
    # a cache whose bytes pass 2^64 still shares them with whatever lies behind its start
    big = dict(paged=paged, int8=int8, H=1024, D=1024, ks=1 << 20, vs=1 << 20, ps=1 << 30, maxp=1, npages=MOST,
               maxlen=MOST, B=2 if paged else MOST)
    assert write(clib, **big, k_new=K + (1 << 30)) == 1 and write(clib, **big, v_new=V + (1 << 30)) == 1
    if paged or int8:
        del big["ks"], big["vs"]
        assert read(clib, **big, n=1, ko=K + (1 << 30)) == 1 and read(clib, **big, n=1, vo=V + (1 << 30)) == 1
