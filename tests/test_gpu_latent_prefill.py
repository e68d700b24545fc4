"""GPU parity of the prefill over expanded latent keys and values against the CPU oracle.

Tolerance as in test_gpu_latent.py (the weights are summed before they are rounded, which the same
bound covers): (2^-8 + 2 e) (sum p |v| + |out|) + 2^-8 |out|, e from the W-product scores."""
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


def make(seed, lens, q_len, H, D, ctx):
    rng = np.random.default_rng(seed)
    B = len(lens)
    draw = lambda *s: f32_to_bf16_bits(rng.standard_normal(s, dtype=np.float32))  # noqa: E731
    c = dict(lens=np.asarray(lens, np.int32), q=draw(B, q_len, H, D + 64), k=draw(B, ctx, H, D), v=draw(B, ctx, H, D),
             pe=draw(B, ctx, 64), scale=float(np.float32((D + 64) ** -0.5)))
    for b, L in enumerate(lens):
        for n in ("k", "v", "pe"):
            c[n][b, max(int(L), 0):] = 0x7FC0  # NaN where no token lies
    return c


def run(c, lens_null=False):
    q = dev_bf16(c["q"])
    out = torch.full((*q.shape[:3], q.shape[3] - 64), float("nan"), dtype=torch.bfloat16, device="cuda")
    binding.latent_prefill_contig(q, dev_bf16(c["k"]), dev_bf16(c["pe"]), dev_bf16(c["v"]),
                                  None if lens_null else dev_i32(c["lens"]), scale=c["scale"], out=out)
    torch.cuda.synchronize()
    assert binding.device_error() == 0
    return host_bits(out)


def check(bits, c, what=""):
    got = values(bits)
    assert np.all(np.isfinite(got)), what
    W = c["q"].shape[-1]
    for b, L in enumerate(c["lens"]):
        L = max(0, min(int(L), c["k"].shape[1]))
        if L == 0:
            assert not got[b].any(), what
            continue
        q, k, v, pe = values(c["q"][b]), values(c["k"][b, :L]), values(c["v"][b, :L]), values(c["pe"][b, :L])
        ref, mass = ol.expanded(q, k, pe, v, c["scale"], spread=True)
        size = abs(c["scale"]) * (np.abs(q).sum(-1).max() * max(np.abs(k).max(), np.abs(pe).max()))
        e = W * 2.0 ** -24 * min(size, 400) + 2.0 ** -21 * 40
        tol = (2.0 ** -8 + 2 * e) * 1.02 * (mass + np.abs(ref)) + 2.0 ** -8 * np.abs(ref) + 1e-30
        bad = np.abs(got[b] - ref) > tol
        assert not bad.any(), (what, b, L, int(bad.sum()), float((np.abs(got[b] - ref) / tol).max()))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("H", [1, 3])
@pytest.mark.parametrize("q_len", [1, 2, 127, 128, 129, 256, 257, 300])
def test_matches_oracle(D, H, q_len):
    # chunk after a prefix, full prefill, chunk longer than the cache (its first queries see nothing), empty
    lens = [q_len + 130, q_len, max(q_len - 5, 1), 0]
    c = make(D + H + q_len, lens, q_len, H, D, q_len + 140)
    check(run(c), c, f"D={D} H={H} q_len={q_len}")


@pytest.mark.parametrize("D", [64, 128])
def test_long_context_and_lengths(D):
    c = make(D, [2000, 1500, 64, 129, 1, 5000, -3], 70, 2, D, 2000)
    c["k"][5], c["v"][5], c["pe"][5] = c["k"][0], c["v"][0], c["pe"][0]  # 5000: clamped to the cache
    check(run(c), c, "lengths")
    c = make(D + 1, [777], 300, 2, D, 777)
    assert np.array_equal(run(c, lens_null=True), run(c))


@pytest.mark.parametrize("D,H,q_len", [(128, 2, 200), (64, 3, 1), (128, 1, 600)])
def test_keys_split_over_parts(D, H, q_len):
    """Few blocks over many key tiles: parts that end within a block's causal border, sequences of one part beside
    sequences of many, empty ones, rows that see nothing of a part."""
    ctx = 2600
    lens = [2600, 511, 513, 0, 1, 2049, q_len // 2 + 1]
    assert binding.load().latent_prefill_workspace_bytes(len(lens), q_len, H, D, ctx, 0) > 0
    c = make(D + q_len, lens, q_len, H, D, ctx)
    first = run(c)
    check(first, c, "parts")
    assert np.array_equal(run(c), first)


@pytest.mark.parametrize("D,H,q_len,lens", [(128, 24, 520, [520, 77, 0, 600]), (64, 40, 300, [300, 0, 512, 130, 700]),
                                            (128, 200, 1, [1, 129]), (64, 320, 3, [2])])
def test_more_blocks_than_multiprocessors(D, H, q_len, lens):
    """CTAs that go on with other CTAs' blocks: blocks of one row tile after two, of one key tile, of none."""
    assert len(lens) * H * -(-q_len // 256) > 152
    c = make(D + H, lens, q_len, H, D, max(lens) + 5)
    first = run(c)
    check(first, c, "blocks")
    args = (dev_bf16(c["q"]), dev_bf16(c["k"]), dev_bf16(c["pe"]), dev_bf16(c["v"]), dev_i32(c["lens"]))
    outs = [torch.full((*args[0].shape[:3], D), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(4)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):  # calls in a row: one's last blocks beside the next one's first
        for out in outs[:3]:
            binding.latent_prefill_contig(*args, scale=c["scale"], out=out)
    graph.replay()
    binding.latent_prefill_contig(*args, scale=c["scale"], out=outs[3])
    torch.cuda.synchronize()
    assert binding.device_error() == 0
    for out in outs:
        assert np.array_equal(host_bits(out), first)


@pytest.mark.parametrize("scale", [-0.1, 0.0, 0.6])
def test_any_scale(scale):
    c = make(9, [400, 200], 200, 2, 128, 400)
    c["scale"] = scale
    check(run(c), c, f"scale={scale}")


def test_rising_scores():
    c = make(10, [700], 256, 2, 64, 700)
    k, q = values(c["k"]), values(c["q"])
    k[..., 0] = np.linspace(0, 30, 700)[None, :, None]
    q[..., 0] = 8.0
    c["k"], c["q"] = f32_to_bf16_bits(k.astype(np.float32)), f32_to_bf16_bits(q.astype(np.float32))
    check(run(c), c, "ramp")


def test_strided_inputs_and_capture():
    """Keys and values as the halves of one expansion, the shared part as the columns of a latent cache."""
    c = make(11, [150, 90], 40, 4, 128, 160)
    for n in ("k", "v", "pe"):
        c[n] = np.where(c[n] == 0x7FC0, 0, c[n]).astype(np.uint16)
    want = run(c)
    kv = torch.cat((dev_bf16(c["k"]), dev_bf16(c["v"])), -1)
    cache = torch.randn(2, 160, 576, device="cuda").to(torch.bfloat16)
    cache[..., 512:] = dev_bf16(c["pe"])
    args = (dev_bf16(c["q"]), kv[..., :128], cache[..., 512:], kv[..., 128:], dev_i32(c["lens"]))
    out = torch.zeros(2, 40, 4, 128, device="cuda", dtype=torch.bfloat16)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        binding.latent_prefill_contig(*args, scale=c["scale"], out=out)
    torch.cuda.synchronize()
    assert np.array_equal(host_bits(out), want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        binding.latent_prefill_contig(*args, scale=c["scale"], out=out)
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert np.array_equal(host_bits(out), want)
    with pytest.raises(ValueError):
        binding.latent_prefill_contig(args[0], kv[..., :128].contiguous(), args[2], kv[..., 128:], scale=1.0)
    one = kv[:1, :1]  # a single token of a single sequence: any strides
    got = binding.latent_prefill_contig(args[0][:1, :1], one[..., :128], cache[:1, :1, 512:], one[..., 128:], scale=1.0)
    assert torch.equal(got[0, 0], one[0, 0, :, 128:])
    none = binding.latent_prefill_contig(args[0], kv[:, :0, :, :128], cache[:, :0, 512:], kv[:, :0, :, 128:], scale=1.0)
    assert not none.any()


def test_absorbed_and_expanded_agree():
    """One model both ways: the expansion's products folded into the queries and the output."""
    rng = np.random.default_rng(12)
    B, n, H, D, R, ctx = 2, 5, 4, 64, 128, 90
    lens = np.array([90, 40], np.int32)
    t = lambda x: torch.from_numpy(x).to("cuda", torch.bfloat16)  # noqa: E731
    cache = t(rng.standard_normal((B, ctx, R + 64)))
    # powers of two and one nonzero a column: the expansion and the absorption are exact in bf16
    up_k = np.zeros((H, D, R))
    up_v = np.zeros((H, D, R))
    for h in range(H):
        up_k[h, np.arange(D), rng.permutation(R)[:D]] = 2.0 ** rng.integers(-1, 2, D)
        up_v[h, np.arange(D), rng.permutation(R)[:D]] = 1.0
    q = t(rng.standard_normal((B, n, H, D + 64)))
    scale = (D + 64) ** -0.5
    c = cache[..., :R].double()
    k = torch.einsum("btr,hdr->bthd", c, torch.from_numpy(up_k).cuda()).to(torch.bfloat16)
    v = torch.einsum("btr,hdr->bthd", c, torch.from_numpy(up_v).cuda()).to(torch.bfloat16)
    exp = binding.latent_prefill_contig(q, k, cache[..., R:], v, dev_i32(lens), scale=scale).double()
    qa = torch.cat((torch.einsum("bihd,hdr->bihr", q[..., :D].double(), torch.from_numpy(up_k).cuda()).to(torch.bfloat16),
                    q[..., D:]), -1).contiguous()
    lat = binding.latent_attn_contig(qa, cache, dev_i32(lens), scale=scale).double()
    absd = torch.einsum("bihr,hdr->bihd", lat, torch.from_numpy(up_v).cuda())
    # each is within (2^-8 + small)(sum p|v| + |out|) + 2^-8 |out| of the same exact value
    kd, vd, pe = k.double().cpu().numpy(), v.double().cpu().numpy(), cache[..., R:].double().cpu().numpy()
    for b, L in enumerate(lens):
        ref, mass = ol.expanded(q[b].double().cpu().numpy(), kd[b, :L], pe[b, :L], vd[b, :L], scale, spread=True)
        tol = (2.0 ** -8 + 1e-3) * 1.02 * (mass + np.abs(ref)) + 2.0 ** -8 * np.abs(ref)
        assert np.all(np.abs(exp[b].cpu().numpy() - ref) <= tol)
        assert np.all(np.abs(absd[b].cpu().numpy() - ref) <= tol)
    assert binding.device_error() == 0


def test_the_capacity_does_not_change_how_keys_are_cut():
    """3000 keys of a cache of that size and of a much larger one: the same parts, so the same bits."""
    H, D, q_len, L, ctx = 8, 128, 200, 3000, 40000
    c = make(14, [L], q_len, H, D, L)
    first = run(c)
    check(first, c, "parts")
    far = [torch.full((1, ctx, *x.shape[2:]), float("nan"), dtype=torch.bfloat16, device="cuda") for x in
           (c["k"], c["pe"], c["v"])]
    for t, n in zip(far, ("k", "pe", "v")):
        t[:, :L] = dev_bf16(c[n])
    out = binding.latent_prefill_contig(dev_bf16(c["q"]), *far, dev_i32(c["lens"]), scale=c["scale"])
    assert np.array_equal(host_bits(out), first)
    assert binding.device_error() == 0


@pytest.mark.parametrize("lens", [[300, 0, 513, 129, -7], [9000, 1, 2, 3, 4]])
def test_launch_groups_by_the_longest_sequence(lens):
    """A capacity that makes several launch groups: every block is still taken exactly once."""
    H, D, q_len, ctx = 11, 128, 300, 8000
    c = make(15, [max(min(L, ctx), 0) for L in lens], q_len, H, D, max(min(max(lens), ctx), 1))
    first = run(c)
    c["lens"] = np.asarray(lens, np.int32)
    if max(lens) <= ctx:
        check(first, c, "groups")
    far = [torch.full((len(lens), ctx, *x.shape[2:]), float("nan"), dtype=torch.bfloat16, device="cuda") for x in
           (c["k"], c["pe"], c["v"])]
    for t, n in zip(far, ("k", "pe", "v")):
        t[:, :c[n].shape[1]] = dev_bf16(c[n])
    out = torch.full((len(lens), q_len, H, D), float("nan"), device="cuda", dtype=torch.bfloat16)
    binding.latent_prefill_contig(dev_bf16(c["q"]), *far, dev_i32(c["lens"]), scale=c["scale"], out=out)
    assert np.array_equal(host_bits(out), first)
    assert binding.device_error() == 0
