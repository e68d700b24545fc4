"""GPU parity of rotary positions, cache writes and cache reads against the CPU oracle,
and the ways they are used: strided, in place, captured, on another stream, with padded
batches, bad pages and full caches; a write, a decode and a read in a row.

Tolerances.  The angle in half turns is an int32 rounded to fp32 (2^-25 half turns at most)
and sincospif is within 2 ulp (2^-23 of 1): cosine and sine are off by pi 2^-25 + 2^-23 + the
float64 phase's 2e-7, under 5e-7; a rotated element a c - b s by (|a| + |b|) magnitude
(5e-7 + 2 2^-24 for its products and sum), and then by half a step of its type."""
import math

import numpy as np
import pytest

from oracle import cache_ops as oc
import oracle
from gqa_split_kv_gb300.workloads import bf16_bits_to_f32, f32_to_bf16_bits

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from gpu_helpers import check_out, dev, dev_bf16, dev_i32, host_bits  # noqa: E402
from gqa_split_kv_gb300 import binding  # noqa: E402

ANGLE = 6.5e-7


def rope_bound(x, ref, w, offset, interleaved, magnitude, eps):
    """Elementwise bound for the rotated heads of x (float64)."""
    n = len(w)
    j = np.arange(n)
    a, b = (offset + 2 * j, offset + 2 * j + 1) if interleaved else (offset + j, offset + n + j)
    mag = np.zeros_like(x)
    mag[..., a] = mag[..., b] = np.abs(x[..., a]) + np.abs(x[..., b])
    return magnitude * mag * ANGLE + np.abs(ref) * eps / 2 * (1 + 1e-6) + 3e-8 * (eps == 2.0 ** -10)


def freqs(rot, base=10000.0):
    return base ** (-2.0 * np.arange(rot // 2) / rot)


# D, rot, offset: whole heads, parts at either end, odd sizes that have no 16-byte chunks
SHAPES = [(128, 128, 0), (256, 64, 0), (192, 64, 128), (64, 32, 16), (40, 24, 8), (10, 6, 3), (3, 2, 1), (96, 96, 0)]


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,rot,offset", SHAPES)
def test_rope_matches_oracle(dtype, interleaved, D, rot, offset):
    rng = np.random.default_rng(D + rot)
    tdt = dict(bf16=torch.bfloat16, f16=torch.float16, f32=torch.float32)[dtype]
    T, H = 37, 5
    x = torch.from_numpy(rng.standard_normal((T, H, D))).to("cuda", tdt)
    pos = rng.integers(-(1 << 31), 1 << 31, T)
    pos[:8] = [0, 1, -1, 2, (1 << 31) - 1, -(1 << 31), 1 << 20, 4097]
    w = freqs(rot)
    xh = x.double().cpu().numpy()
    for backward in (False, True):
        got = binding.rope_apply(x, dev_i32(pos), dev(w), offset=offset, interleaved=interleaved, magnitude=1.25,
                                 backward=backward).double().cpu().numpy()
        ref = oc.rotate(xh, pos, w, offset, interleaved, 1.25, backward)
        # the float64 angle itself is off by 2^-53 of |p w|, on both sides
        far = 2 * np.abs(pos).max() * w.max() * 2.0 ** -52 * 1.25 * 2 * np.abs(xh).max()
        bound = rope_bound(xh, ref, w, offset, interleaved, 1.25, torch.finfo(tdt).eps) + far
        assert np.all(np.abs(got - ref) <= bound), float((np.abs(got - ref) / bound).max())
        rest = np.r_[0:offset, offset + rot:D]
        assert np.array_equal(got[..., rest], xh[..., rest])


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("H,D", [(4, 64), (3, 20)])
def test_rope_strides_and_in_place(interleaved, H, D):
    gen = torch.Generator(device="cuda").manual_seed(D)
    B, n = 3, 5
    fused = torch.randn(B, n, 3 * H * D, generator=gen, device="cuda").to(torch.bfloat16)
    q = fused[..., H * D:2 * H * D].unflatten(-1, (H, D))
    pos = torch.randint(0, 5000, (B, n), generator=gen, device="cuda", dtype=torch.int32)
    w = dev(freqs(D))
    want = binding.rope_apply(q.contiguous(), pos, w, interleaved=interleaved)
    out = torch.full_like(fused, 7.0)
    binding.rope_apply(q, pos, w, interleaved=interleaved, out=out[..., :H * D].unflatten(-1, (H, D)))
    assert torch.equal(out[..., :H * D].unflatten(-1, (H, D)), want) and bool((out[..., H * D:] == 7).all())
    head_major = q.transpose(1, 2).contiguous()[0].transpose(0, 1)  # [n, H, D], heads further apart than tokens
    got = torch.empty_like(head_major)
    assert got.stride() == head_major.stride()
    assert torch.equal(binding.rope_apply(head_major, pos[0], w, interleaved=interleaved, out=got), want[0])
    one = q[:1, :1, :1].expand(1, n, H, D)  # broadcast input: tokens and heads 0 apart
    assert torch.equal(binding.rope_apply(one, pos[:1], w, interleaved=interleaved),
                       binding.rope_apply(one.contiguous(), pos[:1], w, interleaved=interleaved))
    before = fused.clone()
    binding.rope_apply(q, pos, w, interleaved=interleaved, out=q)  # in place, in the fused buffer
    assert torch.equal(q, want)
    keep = torch.ones(3 * H * D, dtype=torch.bool, device="cuda")
    keep[H * D:2 * H * D] = False
    assert torch.equal(fused[..., keep], before[..., keep])
    with pytest.raises(binding.DecodeAttnError):
        binding.rope_apply(fused[..., :H * D].unflatten(-1, (H, D)), pos, w, out=fused[..., 2:H * D + 2].unflatten(-1, (H, D)))


def test_rope_gradient_against_differences_and_autograd_of_the_formula():
    rng = np.random.default_rng(5)
    T, H, D, rot = 6, 2, 24, 16
    w = freqs(rot)
    pos = rng.integers(0, 300, T)
    x, g, d = rng.standard_normal((3, T, H, D)).astype(np.float32)
    gx = binding.rope_apply(dev(g), dev_i32(pos), dev(w), offset=4, magnitude=0.75, backward=True).double().cpu().numpy()
    h = 2.0 ** -6  # the map is linear: differences are exact but for rounding
    up = binding.rope_apply(dev(x + h * d), dev_i32(pos), dev(w), offset=4, magnitude=0.75).double().cpu().numpy()
    dn = binding.rope_apply(dev(x - h * d), dev_i32(pos), dev(w), offset=4, magnitude=0.75).double().cpu().numpy()
    diff = ((up - dn) / (2 * h) * g).sum()
    # rounding: each of the T H D terms off by 4 2^-24 |x| |g| / 2h at most, |x|, |g| under 5
    assert abs(diff - (gx * d).sum()) <= T * H * D * 4 * 2.0 ** -24 * 25 / (2 * h)
    ref = oc.rotate(g.astype(np.float64), pos, w, 4, False, 0.75, True)
    assert np.all(np.abs(gx - ref) <= rope_bound(g.astype(np.float64), ref, w, 4, False, 0.75, 2.0 ** -23))


def test_rope_empty_one_and_many_tokens():
    w = dev(freqs(32))
    for T in (0, 1, 5000):
        x = torch.randn(T, 1, 32, device="cuda")
        pos = torch.arange(T, device="cuda", dtype=torch.int32)
        y = binding.rope_apply(x, pos, w)
        assert y.shape == x.shape
        if T:
            ref = oc.rotate(x.double().cpu().numpy(), pos.cpu().numpy(), freqs(32))
            assert np.abs(y.double().cpu().numpy() - ref).max() < 1e-5 * 5


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,H,D,rot,offset", [(5000, 1, 64, 64, 0), (1301, 3, 40, 24, 8), (2000, 2, 10, 6, 3), (3001, 1, 3, 2, 1),
                                              (4003, 7, 96, 96, 0), (1300, 1, 2048, 2048, 0), (2500, 2, 192, 64, 128)])
def test_rope_many_tokens_of_few_heads(interleaved, dtype, T, H, D, rot, offset):
    """Several tokens a CTA: their number not a multiple of a CTA's, strided, out of place and in place."""
    rng = np.random.default_rng(T)
    tdt = dict(bf16=torch.bfloat16, f32=torch.float32)[dtype]
    wide = torch.from_numpy(rng.standard_normal((T, H + 1, D), dtype=np.float32)).to("cuda", tdt)
    x = wide[:, :H]
    pos = rng.integers(0, 1 << 20, T)
    w = freqs(rot)
    xh = x.double().cpu().numpy()
    ref = oc.rotate(xh, pos, w, offset, interleaved)
    far = 2 * np.abs(pos).max() * w.max() * 2.0 ** -52 * 2 * np.abs(xh).max()
    bound = rope_bound(xh, ref, w, offset, interleaved, 1.0, torch.finfo(tdt).eps) + far
    got = binding.rope_apply(x, dev_i32(pos), dev(w), offset=offset, interleaved=interleaved)
    assert np.all(np.abs(got.double().cpu().numpy() - ref) <= bound)
    last = wide[:, H].clone()
    binding.rope_apply(x, dev_i32(pos), dev(w), offset=offset, interleaved=interleaved, out=x)
    assert torch.equal(x, got) and torch.equal(wide[:, H], last)


# ---------------------------------------------------------------- write and read

def layout(rng, lens, cap, ps):
    """A page table for these lengths and three spare pages; entries past a sequence are -1."""
    need = [-(-min(max(int(L), 0), cap) // ps) for L in lens]
    perm = rng.permutation(sum(need) + 3).astype(np.int32)
    table = np.full((len(lens), -(-cap // ps)), -1, np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
    return table, sum(need) + 3


LENS = [0, 1, 2, 5, 16, 17, 64, 100]


def write_case(seed, B, n, H, D, lens, cap, ps, int8, keys_only=False):
    rng = np.random.default_rng(seed)
    c = dict(lens=np.asarray(lens, np.int32), cap=cap, ps=ps, H=H, D=D, n=n)
    c["new"] = [f32_to_bf16_bits(rng.standard_normal((B, n, H, D), dtype=np.float32)) for _ in "kv"[:1 if keys_only else 2]]
    if ps:
        c["table"], pages = layout(rng, lens, cap, ps)
        lead = (pages, ps)
    else:
        c["table"], lead = None, (B, cap)
    c["cache"], c["scale"] = [], []
    for _ in c["new"]:
        if int8:
            c["cache"].append(rng.integers(-128, 128, (*lead, H, D)).astype(np.int8))
            c["scale"].append(rng.random((lead[0], H, lead[1]), dtype=np.float32))
        else:
            c["cache"].append(f32_to_bf16_bits(rng.standard_normal((*lead, H, D), dtype=np.float32)))
    return c


def to_dev(x):
    return dev(x) if x.dtype == np.int8 else dev_bf16(x)


def run_write(c, w=None, **rope):
    new = [dev_bf16(x) for x in c["new"]]
    cache = [to_dev(x) for x in c["cache"]]
    scale = [dev(x) for x in c["scale"]]
    if len(new) == 1:
        new.append(None), cache.append(None), scale.append(None)
    lens = dev_i32(c["lens"])
    kw = dict(inv_freq=None if w is None else dev(w), **rope)
    s = scale if c["scale"] else []
    if c["ps"]:
        fn = binding.kv_write_int8_paged if s else binding.kv_write_paged
        fn(*new, *cache, *s, dev_i32(c["table"]), lens, c["cap"], **kw)
    else:
        fn = binding.kv_write_int8_contig if s else binding.kv_write_contig
        fn(*new, *cache, *s, lens, **kw)
    torch.cuda.synchronize()
    got = [None if x is None else host_bits(x) if x.dtype == torch.bfloat16 else x.cpu().numpy() for x in cache]
    return got, [None if x is None else x.cpu().numpy() for x in (scale or [None, None])]


def check_write(c, got, scales, w=None, offset=0, interleaved=False, magnitude=1.0):
    late = bad = False
    for i, bits in enumerate(c["new"]):
        x = bf16_bits_to_f32(bits).astype(np.float64)
        rotated = i == 0 and w is not None
        if rotated:
            pos = oc.new_positions(c["lens"], c["n"])
            ref = oc.rotate(x, pos, w, offset, interleaved, magnitude)
            slack = rope_bound(x, ref, w, offset, interleaved, magnitude, 0.0)
        else:
            ref, slack = x, np.zeros_like(x)
        args = (c["lens"], c["cap"], c["table"], c["ps"])
        if not c["scale"]:
            bits_ref = np.asarray(oracle.round_to_bf16(ref))
            want, late, bad = oc.write(c["cache"][i], bits_ref, *args)
            if not rotated:
                assert np.array_equal(got[i], want)
                continue
            where, _, _ = oc.write(np.zeros(c["cache"][i].shape, bool), np.ones(bits.shape, bool), *args)
            assert np.array_equal(got[i][~where], want[~where])
            exact, _, _ = oc.write(np.zeros(c["cache"][i].shape), ref, *args)
            tol, _, _ = oc.write(np.zeros(c["cache"][i].shape), slack + np.abs(ref) * 2.0 ** -8 * (1 + 1e-6), *args)
            err = np.abs(bf16_bits_to_f32(got[i]).astype(np.float64) - exact)
            assert np.all(err[where] <= tol[where])
            continue
        q, s = oc.quantize(ref)
        want, late, bad = oc.write(c["cache"][i], q, *args)
        rows = lambda a: np.ascontiguousarray(np.moveaxis(a, 1, 2))  # scales as [.., tokens, H]  # noqa: E731
        want_s, _, _ = oc.write(rows(c["scale"][i]), s, *args)
        got_s = rows(scales[i])
        if not rotated:
            assert np.array_equal(got[i], want) and np.array_equal(got_s, want_s, equal_nan=True)
            continue
        where, _, _ = oc.write(np.zeros(c["cache"][i].shape[:3], bool), np.ones(bits.shape[:3], bool), *args)
        assert np.array_equal(got[i][~where], want[~where]) and np.array_equal(got_s[~where], want_s[~where])
        exact, _, _ = oc.write(np.zeros(c["cache"][i].shape), ref, *args)
        tol, _, _ = oc.write(np.zeros(c["cache"][i].shape), slack, *args)
        top = tol.max(-1)[where]
        # the scale is a 127th of a maximum that is off by `top`; a value is off by half a step of
        # that scale, the rotation's error and the quotient's rounding (127 2^-24 steps)
        assert np.all(np.abs(got_s - want_s)[where] <= top / 127 + want_s[where] * 2.0 ** -22)
        err = np.abs(got[i].astype(np.float64) * got_s[..., None] - exact)
        lim = got_s[..., None] * (0.5 + 2.0 ** -16) + tol + (tol.max(-1) * 1.01)[..., None]
        assert np.all(err[where] <= lim[where])
    return late, bad


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("ps", [0, 16, 24, 48, 64])
@pytest.mark.parametrize("n,H,D", [(1, 8, 128), (7, 2, 64), (3, 1, 256), (40, 3, 96), (2, 1, 576), (5, 4, 32)])
def test_write_matches_oracle(int8, ps, n, H, D):
    c = write_case(n * D + ps, len(LENS), n, H, D, LENS, 104, ps, int8)
    got, scales = run_write(c)
    check_write(c, got, scales)
    assert binding.device_error() == 0


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,rot,offset", [(128, 128, 0), (128, 64, 64), (256, 32, 8), (64, 16, 24), (576, 64, 512)])
def test_write_rotates_keys(int8, interleaved, D, rot, offset):
    lens = [3, 4100, 4117, 9]  # the first is padded: only its last 3 tokens are written
    c = write_case(D + rot, len(lens), 9, 2, D, lens, 4160, 64, int8)
    w = freqs(rot)
    got, scales = run_write(c, w, offset=offset, interleaved=interleaved, magnitude=1.1)
    check_write(c, got, scales, w, offset, interleaved, 1.1)
    assert binding.device_error() == 0


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("H,D,rot,offset,interleaved", [
    (2, 128, 128, 0, False),   # a pair's halves in one lane's two chunks
    (2, 128, 128, 0, True), (2, 128, 64, 64, False), (1, 64, 64, 0, False), (3, 96, 96, 0, False), (1, 512, 512, 0, False),
    (1, 320, 64, 256, False), (4, 16, 16, 0, False)])
def test_write_many_tokens(int8, H, D, rot, offset, interleaved):
    """Enough tokens that a CTA takes several and a lane two chunks."""
    lens = [700, 650, 20, 900]
    c = write_case(D + H, len(lens), 640, H, D, lens, 912, 16, int8)
    w = freqs(rot)
    got, scales = run_write(c, w, offset=offset, interleaved=interleaved)
    check_write(c, got, scales, w, offset, interleaved)
    got, scales = run_write(c)
    check_write(c, got, scales)
    assert binding.device_error() == 0


@pytest.mark.parametrize("int8", [False, True])
def test_write_keys_only(int8):
    c = write_case(3, 3, 4, 1, 576, [4, 30, 64], 64, 16, int8, keys_only=True)
    got, scales = run_write(c)
    check_write(c, got, scales)


@pytest.mark.parametrize("int8", [False, True])
def test_write_past_the_capacity_and_bad_pages_are_flagged_and_skipped(int8):
    c = write_case(8, 3, 6, 2, 64, [66, 20, 64], 64, 16, int8)  # sequence 0 brings 2 tokens too many
    got, scales = run_write(c)
    late, bad = check_write(c, got, scales)
    assert late and not bad and binding.device_error() == 8
    c = write_case(9, 3, 6, 2, 64, [60, 20, 64], 64, 16, int8)
    c["table"][1, 0], c["table"][1, 1], c["table"][2, 3] = -1, 1 << 30, len(c["cache"][0])
    got, scales = run_write(c)
    late, bad = check_write(c, got, scales)
    assert bad and not late and binding.device_error() == 4
    c = write_case(10, 2, 3, 2, 64, [-5, 2], 40, 0, int8)  # lengths below zero and below the chunk
    got, scales = run_write(c)
    check_write(c, got, scales)
    assert binding.device_error() == 0


def test_write_int8_special_rows():
    """Zeros, ties, subnormal rows, infinities and NaN."""
    D = 64
    rows = np.zeros((6, D), np.float32)
    rows[1, :4] = [1.0, 0.5, -0.5, 0.25]           # 63.5 and -63.5: to even
    rows[2, :2] = [1e-38, 3e-39]                   # a scale below the smallest normal number: floored
    rows[3, 5] = np.inf
    rows[4, 7] = np.nan
    rows[5, :3] = [3.3e38, -3.3e38, 1.0]
    c = write_case(1, 1, 6, 1, D, [6], 16, 16, True)
    c["new"] = [f32_to_bf16_bits(rows).reshape(1, 6, 1, D)] * 2
    c["new"] = [x.copy() for x in c["new"]]
    for x in c["new"]:
        x[0, 4, 0, 7] = 0x7FC0
    got, scales = run_write(c)
    check_write(c, got, scales)


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("H,D,n", [(8, 128, 190), (4, 256, 400), (4, 192, 500), (12, 64, 150), (1, 256, 1700)])
def test_write_many_rows_whole_heads(int8, H, D, n):
    """Rows enough for two or four chunks a lane, whole heads rotated or none, rows with infinities and NaN among them."""
    lens = [n + 3, n - 1]
    c = write_case(D + n, 2, n, H, D, lens, n + 9, 0, int8)
    w = freqs(D)
    got, scales = run_write(c, w)
    check_write(c, got, scales, w)
    if int8:
        c["new"] = [x.copy() for x in c["new"]]
        for x in c["new"]:
            x[0, ::37, 0, D - 1], x[1, ::41, H - 1, 3], x[1, 5] = 0x7F80, 0x7FC0, 0
    got, scales = run_write(c)
    check_write(c, got, scales)
    assert binding.device_error() == 0


def test_write_from_a_fused_projection():
    gen = torch.Generator(device="cuda").manual_seed(4)
    B, n, Hq, H, D = 2, 5, 4, 2, 64
    fused = torch.randn(B, n, (Hq + 2 * H) * D, generator=gen, device="cuda").to(torch.bfloat16)
    k = fused[..., Hq * D:(Hq + H) * D].unflatten(-1, (H, D))
    v = fused[..., (Hq + H) * D:].unflatten(-1, (H, D))
    lens = dev_i32(np.array([5, 9]))
    caches = [torch.zeros(B, 12, H, D, device="cuda", dtype=torch.bfloat16) for _ in range(4)]
    binding.kv_write_contig(k, v, caches[0], caches[1], lens)
    binding.kv_write_contig(k.contiguous(), v.contiguous(), caches[2], caches[3], lens)
    assert torch.equal(caches[0], caches[2]) and torch.equal(caches[1], caches[3])
    assert torch.equal(caches[0][1, 4:9], k[1]) and not caches[0][1, :4].any() and not caches[0][1, 9:].any()


@pytest.mark.parametrize("ps,int8", [(0, True), (16, True), (48, True), (16, False), (40, False)])
@pytest.mark.parametrize("H,D", [(8, 128), (1, 576), (3, 32)])
def test_read_matches_oracle(ps, int8, H, D):
    c = write_case(D + ps, len(LENS), 1, H, D, LENS, 104, ps, int8)
    rng = np.random.default_rng(ps)
    for starts, n in ((None, 104), (rng.integers(-3, 90, len(LENS)).astype(np.int32), 11), (None, 1)):
        before = [f32_to_bf16_bits(rng.standard_normal((len(LENS), n, H, D), dtype=np.float32)) for _ in "kv"]
        out = [dev_bf16(x) for x in before]
        kw = dict(starts=None if starts is None else dev_i32(starts), k_out=out[0], v_out=out[1])
        cache, scale, lens = [to_dev(x) for x in c["cache"]], [dev(x) for x in c["scale"]], dev_i32(c["lens"])
        if ps and int8:
            binding.kv_read_int8_paged(*cache, *scale, dev_i32(c["table"]), lens, 104, n, **kw)
        elif ps:
            binding.kv_read_paged(*cache, dev_i32(c["table"]), lens, 104, n, **kw)
        else:
            binding.kv_read_int8_contig(*cache, *scale, lens, n, **kw)
        for i in range(2):
            ref = oc.read(before[i], c["cache"][i], c["lens"], 104, n, starts, c["table"], ps,
                          c["scale"][i] if int8 else None)
            assert np.array_equal(host_bits(out[i]), ref)
    assert binding.device_error() == 0


def test_read_bad_pages_are_flagged_and_left():
    c = write_case(2, 2, 1, 2, 64, [40, 33], 48, 16, True)
    c["table"][0, 1], c["table"][1, 2] = 999, -7
    before = [f32_to_bf16_bits(np.full((2, 48, 2, 64), 5.0, np.float32)) for _ in "kv"]
    out = [dev_bf16(x) for x in before]
    binding.kv_read_int8_paged(*[dev(x) for x in c["cache"]], *[dev(x) for x in c["scale"]], dev_i32(c["table"]),
                               dev_i32(c["lens"]), 48, 48, k_out=out[0], v_out=out[1])
    for i in range(2):
        assert np.array_equal(host_bits(out[i]), oc.read(before[i], c["cache"][i], c["lens"], 48, 48, None, c["table"],
                                                         16, c["scale"][i]))
    assert binding.device_error() == 4


def test_a_step_in_a_row_captured_and_on_another_stream():
    """Rotate the queries, write the step's keys and values into the int8 pool, decode, read back: against the
    oracle, then captured in a graph and replayed with the next token in the same buffers."""
    rng = np.random.default_rng(11)
    B, Hq, H, D, ps, cap = 5, 8, 2, 64, 16, 96
    lens0 = np.array([1, 16, 17, 40, 90], np.int32)
    c = write_case(12, B, 1, H, D, lens0 + 1, cap, ps, True)
    w = freqs(D)
    state = dict(cache=[dev(x) for x in c["cache"]], scale=[dev(x) for x in c["scale"]], table=dev_i32(c["table"]),
                 lens=dev_i32(lens0), w=dev(w))
    q = torch.zeros(B, Hq, D, device="cuda", dtype=torch.bfloat16)
    new = [torch.zeros(B, 1, H, D, device="cuda", dtype=torch.bfloat16) for _ in "kv"]
    rot, out = torch.empty_like(q), torch.empty_like(q)
    S = binding.num_splits_multi(B, 1, Hq, H, cap, D)
    acc = torch.empty(B, Hq, S, D, device="cuda")
    ml = torch.empty(B, Hq, S, 2, device="cuda")
    ctr = torch.zeros(binding.counters_len(B, Hq, H), dtype=torch.int64, device="cuda")
    back = [torch.zeros(B, cap, H, D, device="cuda", dtype=torch.bfloat16) for _ in "kv"]
    # history: every cached token before the step holds a written row
    prefix = [f32_to_bf16_bits(rng.standard_normal((B, cap, H, D), dtype=np.float32)) for _ in "kv"]
    full = dev_i32(np.full(B, cap))
    wide = np.arange(B * (cap // ps), dtype=np.int32).reshape(B, -1)[:, rng.permutation(cap // ps)]
    state["table"] = dev_i32(wide)
    for k in range(2):
        state["cache"][k] = torch.zeros(B * (cap // ps), ps, H, D, device="cuda", dtype=torch.int8)
        state["scale"][k] = torch.zeros(B * (cap // ps), H, ps, device="cuda")
    binding.kv_write_int8_paged(*[dev_bf16(x) for x in prefix], *state["cache"], *state["scale"], state["table"], full,
                                cap, inv_freq=state["w"])

    def step():
        pos = state["lens"] - 1
        binding.rope_apply(q, pos, state["w"], out=rot)
        binding.kv_write_int8_paged(*new, *state["cache"], *state["scale"], state["table"], state["lens"], cap,
                                    inv_freq=state["w"])
        binding.decode_attn_int8_paged(rot, *state["cache"], *state["scale"], state["table"], state["lens"], cap,
                                       splits=S, part_acc=acc, part_ml=ml, seg_counters=ctr, out=out)
        binding.kv_read_int8_paged(*state["cache"], *state["scale"], state["table"], state["lens"], cap, cap,
                                   k_out=back[0], v_out=back[1])

    def feed(lens):
        qn = f32_to_bf16_bits(rng.standard_normal((B, Hq, D), dtype=np.float32))
        kn = [f32_to_bf16_bits(rng.standard_normal((B, 1, H, D), dtype=np.float32)) for _ in "kv"]
        q.copy_(dev_bf16(qn)), new[0].copy_(dev_bf16(kn[0])), new[1].copy_(dev_bf16(kn[1]))
        state["lens"].copy_(dev_i32(lens))
        return qn

    def check(qn, lens, what):
        torch.cuda.synchronize()
        assert binding.device_error() == 0
        qr = oc.rotate(bf16_bits_to_f32(qn).astype(np.float64), np.asarray(lens) - 1, w)
        inp = dict(q=oracle.round_to_bf16(qr), k_pool_i8=state["cache"][0].cpu().numpy(),
                   v_pool_i8=state["cache"][1].cpu().numpy(), k_scale_pool=state["scale"][0].cpu().numpy(),
                   v_scale_pool=state["scale"][1].cpu().numpy(), page_table=wide, page_size=ps,
                   seq_lens=np.asarray(lens, np.int32), scale=1 / math.sqrt(D))
        check_out(host_bits(out), oracle.decode_int8(inp), what)
        for i, n in enumerate("kv"):
            ref = oc.read(np.zeros((B, cap, H, D), np.uint16), inp[n + "_pool_i8"], lens, cap, cap, None, wide, ps,
                          inp[n + "_scale_pool"])
            got = host_bits(back[i])
            for b, L in enumerate(lens):
                assert np.array_equal(got[b, :L], ref[b, :L])
        # the step's own key, back through the cache: half a step of its scale away
        for b, L in enumerate(lens):
            k = oc.rotate(new[0].double().cpu().numpy()[b], np.array([L - 1]), w)[0]
            got = bf16_bits_to_f32(host_bits(back[0])[b, L - 1]).astype(np.float64)
            lim = np.abs(k).max(-1, keepdims=True) / 254 * 1.01 + np.abs(k) * 2.0 ** -8 * 1.01 + 1e-5
            assert np.all(np.abs(got - k) <= lim)

    qn = feed(lens0 + 1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    check(qn, lens0 + 1, "on another stream")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for more in (2, 3):
        qn = feed(lens0 + more)
        graph.replay()
        check(qn, lens0 + more, f"replayed {more}")


@pytest.mark.parametrize("tokens", [3, 2500])
def test_calls_in_a_row_see_each_other(tokens):
    """Every kernel may start while the one before it drains: dependent calls queued without a pause, torch's
    own kernels among them, give what the same calls give one at a time."""
    gen = torch.Generator(device="cuda").manual_seed(tokens)
    H, D, R, ps = 2, 64, 128, 16
    pages = -(-tokens // ps)
    w, w64 = binding.rope_inv_freq(D), binding.rope_inv_freq(64)
    table = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)[None]
    start = torch.randn(1, tokens, H, D, generator=gen, device="cuda").to(torch.bfloat16)
    qs = torch.randn(1, 1, 8, R + 64, generator=gen, device="cuda").to(torch.bfloat16)

    def chain(pause):
        x, lens = start.clone(), torch.zeros(1, dtype=torch.int32, device="cuda")
        pos = torch.zeros(1, tokens, dtype=torch.int32, device="cuda")
        pool = [torch.zeros(pages, ps, H, D, dtype=torch.int8, device="cuda") for _ in "kv"]
        scale = [torch.zeros(pages, H, ps, device="cuda") for _ in "kv"]
        latent = torch.zeros(pages, ps, R + 64, dtype=torch.bfloat16, device="cuda")
        seen = []
        for i in range(12):
            pos.fill_(i * 1000).add_(torch.arange(tokens, device="cuda", dtype=torch.int32))
            lens.fill_(tokens)
            pause()
            binding.rope_apply(x, pos, w, out=x)
            pause()
            binding.kv_write_int8_paged(x, x, *pool, *scale, table, lens, tokens, inv_freq=w)
            pause()
            k, v = binding.kv_read_int8_paged(*pool, *scale, table, lens, tokens, tokens)
            pause()
            binding.rope_apply(k, pos, w, backward=True, out=x)
            pause()
            row = torch.cat((x.flatten(2), v.flatten(2)[..., :64]), -1)[:, :, None]
            binding.kv_write_paged(row, None, latent[:, :, None], None, table, lens, tokens, inv_freq=w64, offset=R)
            pause()
            out = binding.latent_attn_paged(qs, latent, table, lens, tokens, scale=0.1)
            pause()
            x.mul_(1.0 + out.float().mean().clamp(-0.1, 0.1).to(torch.bfloat16))
            lens.zero_()  # after the calls that read it
            seen.append(x.clone())
        torch.cuda.synchronize()
        return torch.stack(seen)

    slow = chain(torch.cuda.synchronize)
    for _ in range(5):
        assert torch.equal(chain(lambda: None), slow)
    assert binding.device_error() == 0


def test_offsets_past_32_bits():
    """A pool of over 2^32 bytes and 2^31 elements: its last pages written, attended to and read; heads far apart."""
    W, ps, pages = 576, 64, 66000  # 2.4e9 elements, 4.9 GB
    pool = torch.zeros(pages, ps, W, device="cuda", dtype=torch.bfloat16)
    gen = torch.Generator(device="cuda").manual_seed(1)
    L = 150
    rows = torch.randn(1, L, 1, W, generator=gen, device="cuda").to(torch.bfloat16)
    table = torch.tensor([[pages - 1, pages - 3, pages - 2]], dtype=torch.int32, device="cuda")
    lens = dev_i32(np.array([L]))
    binding.kv_write_paged(rows, None, pool[:, :, None], None, table, lens, 192)
    back, _ = binding.kv_read_paged(pool[:, :, None], None, table, lens, 192, L)
    assert torch.equal(back, rows)
    q = torch.randn(1, 1, 16, W, generator=gen, device="cuda").to(torch.bfloat16)
    small = binding.latent_attn_contig(q, rows[:, :, 0].contiguous(), scale=0.05)
    assert torch.equal(binding.latent_attn_paged(q, pool, table, lens, 192, scale=0.05), small)
    assert int((pool.view(torch.int16)[: pages - 3] != 0).sum()) == 0
    k8 = pool.view(torch.int8).view(pages, ps, 2, W)  # the same memory as an int8 pool
    scale = torch.zeros(pages, 2, ps, device="cuda")
    new = torch.randn(1, L, 2, W, generator=gen, device="cuda").to(torch.bfloat16)
    binding.kv_write_int8_paged(new, None, k8, None, scale, None, table, lens, 192)
    back, _ = binding.kv_read_int8_paged(k8, None, scale, None, table, lens, 192, L)
    near, near_scale = torch.zeros(1, 192, 2, W, device="cuda", dtype=torch.int8), torch.zeros(1, 2, 192, device="cuda")
    binding.kv_write_int8_contig(new, None, near, None, near_scale, None, lens)
    want, _ = binding.kv_read_int8_contig(near, None, near_scale, None, lens, L)
    assert torch.equal(back, want) and bool(want.any())
    x = pool.view(-1)
    far = torch.as_strided(x, (2, 2, 64), (2 ** 30 + 2 ** 29, 2 ** 29, 1))
    far.copy_(torch.randn(2, 2, 64, generator=gen, device="cuda"))
    pos, w = dev_i32(np.array([5, 1000])), binding.rope_inv_freq(64)
    want = binding.rope_apply(far.contiguous(), pos, w)
    binding.rope_apply(far, pos, w, out=far)
    assert torch.equal(far, want)


def test_empty_caches():
    """A cache of no pages or no tokens: nothing is read, a written token is flagged."""
    bf16, z = torch.bfloat16, dev_i32(np.array([0, 0]))
    pool, table = torch.zeros(0, 16, 2, 64, device="cuda", dtype=bf16), torch.zeros(2, 3, device="cuda", dtype=torch.int32)
    k, v = binding.kv_read_paged(pool, pool.clone(), table, dev_i32(np.array([5, 0])), 48, 4)
    assert not k.any() and not v.any() and binding.device_error() == 0
    new = torch.ones(2, 1, 2, 64, device="cuda", dtype=bf16)
    binding.kv_write_paged(new, new, pool, pool.clone(), table, z, 48)  # lengths 0: nothing to write
    assert binding.device_error() == 0
    binding.kv_write_paged(new, new, pool, pool.clone(), table, dev_i32(np.array([1, 0])), 48)
    assert binding.device_error() == 4
    cache = torch.zeros(2, 0, 2, 64, device="cuda", dtype=bf16)
    binding.kv_write_contig(new, new, cache, cache.clone(), dev_i32(np.array([1, 0])))
    assert binding.device_error() == 8
    q = torch.ones(2, 1, 4, 192, device="cuda", dtype=bf16)
    assert not binding.latent_attn_contig(q, torch.zeros(2, 0, 192, device="cuda", dtype=bf16), scale=1.0).any()


FIRST_CALL_CAPTURED = """
import torch
from gqa_split_kv_gb300 import binding
bf16 = torch.bfloat16
gen = torch.Generator(device="cuda").manual_seed(3)
x = torch.randn(8, 2, 64, generator=gen, device="cuda").to(bf16)
pos = torch.arange(8, device="cuda", dtype=torch.int32)
w = (10000.0 ** (-torch.arange(32, dtype=torch.float64) / 32)).cuda()
new = torch.randn(2, 4, 2, 64, generator=gen, device="cuda").to(bf16)
k = torch.zeros(2, 8, 2, 64, device="cuda", dtype=torch.int8)
ks = torch.zeros(2, 2, 8, device="cuda")
lens = torch.tensor([4, 8], device="cuda", dtype=torch.int32)
q = torch.randn(2, 1, 4, 192, generator=gen, device="cuda").to(bf16)
cache = torch.randn(2, 8, 192, generator=gen, device="cuda").to(bf16)
qe = torch.randn(2, 3, 2, 128, generator=gen, device="cuda").to(bf16)
kv = torch.randn(2, 600, 2, 128, generator=gen, device="cuda").to(bf16)
pe = torch.randn(2, 600, 64, generator=gen, device="cuda").to(bf16)

def calls():
    a = binding.rope_apply(x, pos, w)
    v, vs = k.clone(), ks.clone()
    binding.kv_write_int8_contig(new, new, k, v, ks, vs, lens, inv_freq=w)
    b, c = binding.kv_read_int8_contig(k, v, ks, vs, lens, 8)
    d = binding.latent_attn_contig(q, cache, lens, scale=0.1)
    e = binding.latent_prefill_contig(qe, kv[..., :64], pe, kv[..., 64:], scale=0.1)
    return a, b, c, d, e

graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = calls()
graph.replay()
torch.cuda.synchronize()
for g, r in zip(got, calls()):
    assert torch.equal(g, r)
assert binding.device_error() == 0
print("first calls captured")
"""


def test_the_first_calls_of_a_process_may_be_captured():
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    res = subprocess.run([sys.executable, "-c", FIRST_CALL_CAPTURED], cwd=root, capture_output=True, text=True, timeout=300)
    assert res.returncode == 0 and "first calls captured" in res.stdout, res.stdout + res.stderr
