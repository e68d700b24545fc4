"""GPU parity of latent attention (absorbed form) against the CPU oracle, and the ways it is used.

Tolerance.  A weight is off by its rounding to bf16 (2^-8 of it at most) and by its score's error e:
fp32 sums of W products (W 2^-24 scale sum |q c|), the scale's rounding and exp2 (2^-21 of a score
under 40).  The weights are summed as rounded, so out = sum w' c / sum w' moves by at most
(2^-8 + 2 e) (sum p |c| + |out|), and is then rounded to bf16 (2^-8 of it)."""
import math

import numpy as np
import pytest

from oracle import latent_attention as ol
from gqa_split_kv_gb300.workloads import bf16_bits_to_f32, f32_to_bf16_bits

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from gpu_helpers import dev_bf16, dev_i32, host_bits  # noqa: E402
from gqa_split_kv_gb300 import binding  # noqa: E402


def values(bits):
    return bf16_bits_to_f32(bits).astype(np.float64)


def make(seed, lens, q_len, H, R, cap, ps=0, spread=1.0):
    rng = np.random.default_rng(seed)
    B, W = len(lens), R + 64
    c = dict(lens=np.asarray(lens, np.int32), R=R, cap=cap, ps=ps, scale=float(np.float32(spread / math.sqrt(W / 3))))
    c["q"] = f32_to_bf16_bits(rng.standard_normal((B, q_len, H, W), dtype=np.float32))
    rows = f32_to_bf16_bits(rng.standard_normal((B, cap, W), dtype=np.float32))
    c["rows"] = rows
    if ps:
        need = [-(-min(max(int(L), 0), cap) // ps) for L in lens]
        perm = rng.permutation(sum(need) + 2).astype(np.int32)
        c["table"] = np.full((B, -(-cap // ps)), -1, np.int32)
        c["pool"] = np.full((sum(need) + 2, ps, W), 0x7FC0, np.uint16)  # NaN where no token lies
        at = 0
        for b, n in enumerate(need):
            c["table"][b, :n] = perm[at:at + n]
            at += n
            for j in range(n):
                t0, t1 = j * ps, min(int(lens[b]), (j + 1) * ps, cap)
                c["pool"][c["table"][b, j], :t1 - t0] = rows[b, t0:t1]
    else:
        for b, L in enumerate(lens):
            rows[b, max(int(L), 0):] = 0x7FC0
    return c


def run(c, lens_null=False, **kw):
    q = dev_bf16(c["q"])
    out = torch.full((*q.shape[:3], c["R"]), float("nan"), dtype=torch.bfloat16, device="cuda")
    lens = None if lens_null else dev_i32(c["lens"])
    if c["ps"]:
        binding.latent_attn_paged(q, dev_bf16(c["pool"]), dev_i32(c["table"]), lens, c["cap"], scale=c["scale"],
                                  out=out, **kw)
    else:
        binding.latent_attn_contig(q, dev_bf16(c["rows"]), lens, scale=c["scale"], out=out, **kw)
    torch.cuda.synchronize()
    return host_bits(out)


def check(bits, c, what="", sequences=None):
    got = values(bits)
    assert np.all(np.isfinite(got)), what
    W = c["R"] + 64
    for b, L in enumerate(c["lens"]):
        if sequences is not None and b not in sequences:
            continue
        L = max(0, min(int(L), c["cap"]))
        q, rows = values(c["q"][b]), values(c["rows"][b, :L])
        if L == 0:
            assert not got[b].any(), what
            continue
        ref, mass = ol.absorbed(q, rows, c["R"], c["scale"], spread=True)
        size = np.abs(c["scale"]) * np.einsum("ihw,tw->iht", np.abs(q), np.abs(rows)).max()
        e = W * 2.0 ** -24 * size + 2.0 ** -21 * 40
        tol = (2.0 ** -8 + 2 * e) * 1.02 * (mass + np.abs(ref)) + 2.0 ** -8 * np.abs(ref) + 1e-30
        bad = np.abs(got[b] - ref) > tol
        assert not bad.any(), (what, b, int(L), int(bad.sum()), float((np.abs(got[b] - ref) / tol).max()))


LENS = [0, 1, 2, 63, 64, 65, 130, 200, 1000]


@pytest.mark.parametrize("R", [128, 256, 512])
@pytest.mark.parametrize("H", [1, 16, 17, 33, 64, 128])
def test_contig_matches_oracle(R, H):
    c = make(R + H, LENS, 1, H, R, 1001)
    check(run(c), c, f"R={R} H={H}")
    assert binding.device_error() == 0


@pytest.mark.parametrize("R,H", [(512, 16), (512, 64), (256, 20), (128, 100)])
@pytest.mark.parametrize("ps", [16, 32, 48, 64, 80, 96, 128])
def test_paged_matches_contiguous_bitwise(R, H, ps):
    c = make(R + H, LENS, 1, H, R, 1001)
    p = make(R + H, LENS, 1, H, R, 1001, ps)
    assert np.array_equal(c["q"], p["q"])
    first = run(p)
    check(first, p, f"ps={ps}")
    assert np.array_equal(first, run(c))
    assert binding.device_error() == 0


@pytest.mark.parametrize("R,H,q_len", [(512, 16, 2), (512, 128, 3), (256, 5, 16), (128, 8, 7), (512, 1, 16), (256, 40, 4)])
@pytest.mark.parametrize("ps", [0, 32])
def test_several_new_tokens(R, H, q_len, ps):
    lens = [q_len, q_len + 1, max(q_len - 2, 0), 0, 1, 64 + q_len // 2, 300]  # some queries see nothing
    c = make(7 * R + H, lens, q_len, H, R, 320, ps)
    check(run(c), c, f"R={R} H={H} q_len={q_len}")
    assert binding.device_error() == 0


@pytest.mark.parametrize("H", [16, 64])
@pytest.mark.parametrize("L", [1, 64, 4096, 20001])
def test_one_sequence_over_many_pieces(H, L):
    c = make(H + L, [L], 1, H, 512, L)
    check(run(c), c, f"L={L}")
    check(run(c, lens_null=True), c, f"L={L}, no lengths")


@pytest.mark.parametrize("scale", [-0.07, 0.0, 1.0])
def test_any_scale(scale):
    # 1.0: scores spread over +-60, so the reference maximum is raised over and over
    c = make(5, [700, 64, 333], 2, 24, 256, 700)
    c["scale"] = scale
    check(run(c), c, f"scale={scale}")


def test_rising_scores_and_outliers():
    """Scores that grow with the position (the running maximum is raised in most tiles) and a late outlier."""
    c = make(6, [900, 640], 1, 16, 128, 900)
    rows = values(c["rows"])
    ramp = np.linspace(0.1, 12.0, 900)
    rows[:, :, 0] = ramp
    rows[1, 600] *= 20
    c["rows"] = f32_to_bf16_bits(np.nan_to_num(rows).astype(np.float32))
    q = values(c["q"])
    q[..., 0] = 12.0
    c["q"] = f32_to_bf16_bits(q.astype(np.float32))
    check(run(c), c, "ramp")


def test_lengths_beyond_the_cache_and_negative_are_clamped():
    c = make(8, [100, 3, 50], 1, 16, 128, 100)
    c["rows"][1:] = c["rows"][0]
    c["lens"] = np.array([5000, -4, 100], np.int32)
    check(run(c), c, "clamped")


@pytest.mark.parametrize("H", [8, 64])
def test_many_sequences(H):
    rng = np.random.default_rng(3)
    lens = np.clip(np.exp(rng.uniform(0, np.log(400), 700)), 0, 400).astype(np.int32)
    lens[::50] = 0
    c = make(9, lens, 1, H, 128, 400, 16)
    check(run(c), c, "700 sequences", sequences=range(0, 700, 23))
    assert binding.device_error() == 0


def test_batch_limit_and_workspace_refusals():
    n = binding.latent_max_batch(1, 128)
    lens = np.full(n, 3, np.int32)
    lens[::3] = 0
    c = make(10, lens, 1, 1, 128, 3)
    check(run(c), c, "batch limit", sequences=[0, 1, 2, n // 2, n - 2, n - 1])
    q = torch.zeros(n + 1, 1, 1, 192, device="cuda", dtype=torch.bfloat16)
    with pytest.raises(binding.DecodeAttnError):
        binding.latent_attn_contig(q, torch.zeros(n + 1, 4, 192, device="cuda", dtype=torch.bfloat16), scale=1.0)
    small = binding.latent_workspace(4, 1, 128)[:-16]
    with pytest.raises(binding.DecodeAttnError):
        binding.latent_attn_contig(q[:4], torch.zeros(4, 4, 192, device="cuda", dtype=torch.bfloat16), scale=1.0,
                                   workspace=small)


def test_bad_page_is_flagged_and_reads_page_zero():
    c = make(11, [100, 40], 1, 16, 256, 112, 16)
    c["pool"][:] = np.where(c["pool"] == 0x7FC0, 0, c["pool"])
    c["table"][0, 3] = 12345
    c["rows"][0, 48:64] = c["pool"][0]
    check(run(c), c, "bad page")
    assert binding.device_error() == 4


def test_reproducible_and_captured_and_on_another_stream():
    c = make(12, [3000, 17, 900, 0, 1], 1, 40, 512, 3000)
    first = run(c)
    work = binding.latent_workspace(5, 40, 512)
    for _ in range(2):
        work.fill_(255)  # any content: NaN
        assert np.array_equal(run(c, workspace=work), first)
    q, rows, lens = dev_bf16(c["q"]), dev_bf16(c["rows"]), dev_i32(c["lens"])
    out = torch.zeros(5, 1, 40, 512, device="cuda", dtype=torch.bfloat16)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        binding.latent_attn_contig(q, rows, lens, scale=c["scale"], workspace=work, out=out)
    torch.cuda.synchronize()
    assert np.array_equal(host_bits(out), first)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        binding.latent_attn_contig(q, rows, lens, scale=c["scale"], workspace=work, out=out)
    for new in ([3000, 17, 900, 0, 1], [5, 3000, 0, 64, 2999], [0, 0, 0, 0, 0]):
        d = dict(c, lens=np.asarray(new, np.int32))
        full = make(12, [3000] * 5, 1, 40, 512, 3000)  # the same draw, with every row present
        rows.copy_(dev_bf16(full["rows"]))
        d["rows"] = full["rows"]
        lens.copy_(dev_i32(d["lens"]))
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        check(host_bits(out), d, f"replayed {new}")
    assert binding.device_error() == 0


def test_row_with_one_heavy_token_is_that_token():
    """One score far above the rest: the weights are summed as rounded, so the output is the token's latent."""
    c = make(13, [300], 1, 16, 128, 300)
    rows = np.zeros((1, 300, 192), np.float32)
    rows[0, :, :128] = np.random.default_rng(1).standard_normal((300, 128))
    rows[0, 211, 128] = 50.0
    q = np.zeros((1, 1, 16, 192), np.float32)
    q[..., 128] = 30.0
    c["rows"], c["q"], c["scale"] = f32_to_bf16_bits(rows), f32_to_bf16_bits(q), 0.37
    assert np.array_equal(run(c)[0, 0], np.repeat(c["rows"][:1, 211, :128], 16, 0))


def test_write_attend_read_over_a_latent_pool():
    """Two steps over one paged pool: write the rows (rotating their shared part), attend, read them back; the
    absorbed result equals the expanded attention that the oracle computes from the same rows."""
    rng = np.random.default_rng(21)
    B, H, R, D, ps, cap = 3, 8, 128, 32, 16, 96
    W = R + 64
    lens = np.array([40, 1, 77], np.int32)
    pool = torch.zeros(20, ps, W, device="cuda", dtype=torch.bfloat16)
    table = dev_i32(rng.permutation(20)[:18].reshape(3, 6))
    w = binding.rope_inv_freq(64)
    new = torch.from_numpy(rng.standard_normal((B, cap, 1, W))).to("cuda", torch.bfloat16)
    binding.kv_write_paged(new, None, pool.unsqueeze(2), None, table, dev_i32(lens), cap, inv_freq=w, offset=R)
    rows, _ = binding.kv_read_paged(pool.unsqueeze(2), None, table, dev_i32(lens), cap, cap)
    rows = rows[:, :, 0].double().cpu().numpy()
    up = rng.standard_normal((H, D, R)) / math.sqrt(R)      # k_nope[t, h] = up[h] c_t
    q_nope, q_rope = rng.standard_normal((B, 1, H, D)), rng.standard_normal((B, 1, H, 64))
    q = np.concatenate([np.einsum("bihd,hdr->bihr", q_nope, up), q_rope], -1)
    qb = torch.from_numpy(q).to("cuda", torch.bfloat16)
    scale = (D + 64) ** -0.5
    out = binding.latent_attn_paged(qb, pool, table, dev_i32(lens), cap, scale=scale).double().cpu().numpy()
    qv = qb.double().cpu().numpy()
    for b, L in enumerate(lens):
        c = rows[b, :L]
        ref, mass = ol.absorbed(qv[b], c, R, scale, spread=True)
        size = scale * np.einsum("ihw,tw->iht", np.abs(qv[b]), np.abs(c)).max()
        tol = (2.0 ** -8 + 2 * (W * 2.0 ** -24 * size + 2e-5)) * 1.02 * (mass + np.abs(ref)) + 2.0 ** -8 * np.abs(ref)
        assert np.all(np.abs(out[b] - ref) <= tol)
        # expanded: keys and values per head from the same rows (values: the latent itself)
        k = np.einsum("tr,hdr->thd", c[:, :R], up)
        pe = np.einsum("ihd,thd->iht", q_nope[b], k) + np.einsum("ihd,td->iht", q_rope[b], c[:, R:])
        p = np.exp(scale * (pe - pe.max(-1, keepdims=True)))
        p /= p.sum(-1, keepdims=True)
        exp = np.einsum("iht,tr->ihr", p, c[:, :R])
        # the absorbed query was rounded to bf16: a score moves by 2^-8 scale sum |q c| at most
        move = 2 * 2.0 ** -8 * size
        assert np.all(np.abs(out[b] - exp) <= tol + np.expm1(move) * (mass + np.abs(ref)))
    assert binding.device_error() == 0
