"""GPU parity of attention weights and eviction against the CPU oracle, and the two with decode."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from long_cache_helpers import Cache, check_attention, f64, lens_of, randn, score_error  # noqa: E402
from oracle import long_cache as ol  # noqa: E402
from gqa_split_kv_gb300 import binding  # noqa: E402


def weigh(c, q, prior, **kw):
    """kv_weights_* of the cache's kind; prior and out as pools where it is paged."""
    if c.int8:
        if c.page:
            return binding.kv_weights_int8_paged(q, c.kp, c.ksp, prior, c.table, c.seq_lens, c.cap, **kw)
        return binding.kv_weights_int8_contig(q, c.k, c.ks, prior, c.seq_lens, **kw)
    if c.page:
        return binding.kv_weights_paged(q, c.kp, prior, c.table, c.seq_lens, c.cap, **kw)
    return binding.kv_weights_contig(q, c.k, prior, c.seq_lens, **kw)


def check_weights(c, q, got, prior, decay=1.0, scale=None):
    D = q.shape[-1]
    scale = D ** -0.5 if scale is None else scale
    rows = q.shape[1] * q.shape[2] // c.H
    for b, L in enumerate(c.live):
        if L == 0:
            continue
        k = c.values("k", b)
        w = ol.weights(f64(q[b]), k, scale)
        before = decay * f64(prior[b, :, :L]) if prior is not None else 0.0
        # a weight moves by twice its score's error; sums of `rows` terms and of the row's own, in fp32
        tol = w * (2 * score_error(f64(q[b]), k, scale, D) + (rows + 64) * 2.0 ** -24) + 2.0 ** -22 * (np.abs(before) + w) \
            + rows * 1e-37
        err = np.abs(f64(got[b, :, :L]) - (w + before))
        assert (err <= tol).all(), (b, L, err.max())


@pytest.mark.parametrize("page", [0, 16, 48])
@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("D,Hq,Hkv", [(64, 8, 4), (128, 8, 2), (256, 6, 1), (128, 40, 1)])
@pytest.mark.parametrize("lens,n", [([0, 1, 64, 65, 700], 1), ([3, 0, 300], 4), ([200, 20], 25)])
def test_weights(page, int8, D, Hq, Hkv, lens, n):
    c = Cache(D + n, lens, max(lens) + 20, Hkv, D, page, names="k", int8=int8)
    c.put_numbers("w", torch.rand(c.B, Hkv, c.cap, generator=c.gen, device="cuda") * 3)
    q = randn(c.gen, c.B, n, Hq, D)
    prior = c.wp if page else c.w
    out = torch.full_like(prior, 9.0)
    assert weigh(c, q, prior, out=out, decay=0.75) is out
    check_weights(c, q, c.numbers_back(out) if page else out, c.w, 0.75)
    touched = sum(c.live) * Hkv
    assert int((out != 9).sum()) == touched  # nothing past a sequence
    other = prior.clone()
    assert weigh(c, q, other) is other
    assert torch.equal(torch.isnan(other), torch.isnan(prior))
    check_weights(c, q, c.numbers_back(other) if page else other, c.w)
    made = weigh(c, q, None)
    check_weights(c, q, c.numbers_back(made) if page else made, None)
    assert binding.device_error() == 0


@pytest.mark.parametrize("int8", [False, True])
def test_weights_of_long_sequences(int8):
    c = Cache(8, [9000, 1, 5000, 8191], 9001, 2, 128, 32, names="k", int8=int8)
    q = randn(c.gen, 4, 1, 8, 128)
    check_weights(c, q, c.numbers_back(weigh(c, q, None)), None)
    c = Cache(9, [20000], 20000, 1, 128, 0, names="k", int8=int8)
    q = randn(c.gen, 1, 64, 16, 128)  # the largest number of rows
    check_weights(c, q, weigh(c, q, None), None)
    total = weigh(c, q, None).double().sum()
    assert abs(float(total) - 1024) < 1024 * 2.0 ** -12


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("rows", [1, 3, 5, 7, 9, 11, 15, 17, 33])
def test_weights_of_any_number_of_rows(rows, D, int8):
    c = Cache(rows, [130, 0, 1, 513], 600, 2, D, 16, names="k", int8=int8)
    q = randn(c.gen, 4, 1, 2 * rows, D)
    check_weights(c, q, c.numbers_back(weigh(c, q, None)), None)


@pytest.mark.parametrize("page", [0, 32])
@pytest.mark.parametrize("n,Hq,D", [(1, 8, 128), (2, 16, 256), (40, 8, 64), (40, 8, 128), (20, 10, 256)])
def test_weights_of_growing_scores(n, Hq, D, page):
    """The largest score comes late and the sums pass every limit of a running maximum on the way."""
    c = Cache(n, [3000, 900, 2048], 3000, 2, D, page, names="k")
    grow = torch.linspace(0.1, 9, 3000, device="cuda")
    c.k.mul_(grow.view(1, 3000, 1, 1))
    if page:
        for b, L in enumerate(c.lens):
            for t in range(0, L, page):
                c.kp[int(c.table[b, t // page]), :min(page, L - t)] = c.k[b, t:min(t + page, L)]
    q = randn(c.gen, 3, n, Hq, D) * 3
    got = weigh(c, q, None)
    check_weights(c, q, c.numbers_back(got) if page else got, None)


def numbers(c, seed, kind):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    w = torch.rand(c.B, c.H, c.cap, generator=gen, device="cuda") ** 6
    if kind == "zeros":
        w = torch.where(torch.rand(w.shape, generator=gen, device="cuda") < 0.9, torch.zeros_like(w), w)
    elif kind == "few":
        w = (w * 4).floor() / 4 - 0.25
    elif kind == "special":
        r = torch.rand(w.shape, generator=gen, device="cuda")
        for at, x in enumerate((float("nan"), float("inf"), -float("inf"), -0.0, 0.0, 1e-42, -3.0)):
            w = torch.where((r > at * 0.1) & (r < at * 0.1 + 0.1), torch.full_like(w, x), w)
    c.put_numbers("w", w)


def evict(c, keep, first, recent, to=None):
    """In place, or to contiguous outputs with `to` rows; returns kept, new_lens and the moved tensors, contiguous."""
    kw, out = dict(first=first, recent=recent), {}
    if to is not None:
        out = dict(k_out=torch.full((c.B, to, c.H, c.D), 3, device="cuda").to(c.k.dtype))
        out["v_out"] = out["k_out"].clone()
        if c.int8:
            out["k_scale_out"] = torch.full((c.B, c.H, to), 5.0, device="cuda")
            out["v_scale_out"] = out["k_scale_out"].clone()
        out["weights_out"] = torch.full((c.B, c.H, to), 5.0, device="cuda")
    p = "p" if c.page else ""
    args = [getattr(c, x + p) for x in (("k", "v", "ks", "vs", "w") if c.int8 else ("k", "v", "w"))]
    pages = (c.table, c.seq_lens, c.cap) if c.page else (c.seq_lens,)
    name = "kv_evict" + ("_int8" if c.int8 else "") + ("_paged" if c.page else "_contig")
    kept, new_lens = getattr(binding, name)(*args, *pages, keep, **kw, **out)
    if to is not None:
        return kept, new_lens, [out[x] for x in out]
    if c.page:
        return kept, new_lens, [c.rows_back(x) if x.dim() == 4 else c.numbers_back(x) for x in args]
    return kept, new_lens, args


@pytest.mark.parametrize("page", [0, 16, 20])
@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("kind", ["plain", "zeros", "few", "special"])
@pytest.mark.parametrize("lens,keep,first,recent", [([0, 1, 50, 51, 52, 3000], 50, 4, 16), ([1500, 2049], 1024, 0, 0),
                                                    ([700, 30], 20, 4, 16), ([333], 1, 0, 1)])
def test_eviction(page, int8, in_place, kind, lens, keep, first, recent):
    c = Cache(keep, lens, max(lens) + 9, 3, 32, page, int8=int8)
    numbers(c, keep, kind)
    names = ("k", "v", "ks", "vs", "w") if int8 else ("k", "v", "w")
    before = {x: getattr(c, x).clone() for x in names}
    kept, new_lens, moved = evict(c, keep, first, recent, None if in_place else keep + 3)
    assert new_lens.tolist() == [min(L, keep) for L in lens]
    for b, L in enumerate(lens):
        n = min(L, keep)
        for h in range(c.H):
            want = ol.evict(f64(before["w"][b, h, :L]), keep, first, recent)
            assert (kept[b, h].cpu().numpy() == np.concatenate((want, np.full(keep - n, -1)))).all(), (b, h)
            at = torch.from_numpy(want).cuda()
            for x, y in zip(names, moved):
                if x in "kv":
                    assert torch.equal(y[b, :n, h], before[x][b, at, h])
                    rest, old = y[b, n:, h], (before[x][b, n:, h] if in_place else torch.full_like(y[b, n:, h], 3))
                    keep_rest = L if in_place and page else None  # past a sequence's pages there is nothing to compare
                    assert torch.equal(rest[:None if keep_rest is None else keep_rest - n].view(torch.int8),
                                       old[:None if keep_rest is None else keep_rest - n].view(torch.int8))
                else:
                    assert torch.equal(y[b, h, :n].view(torch.int32), before[x][b, h, at].view(torch.int32))
            if in_place:
                assert not moved[-1][b, h, n:L].any()
            else:
                assert not moved[-1][b, h, n:].any()
    assert binding.device_error() == 0


def test_keys_alone_and_wide_rows():
    for D, int8 in ((576, False), (1024, True), (16, True)):
        c = Cache(D, [500, 90], 500, 1, D, 16, names="k", int8=int8)
        numbers(c, D, "plain")
        if int8:
            kept, _ = binding.kv_evict_int8_paged(c.kp, None, c.ksp, None, c.wp, c.table, c.seq_lens, c.cap, 70)
        else:
            kept, _ = binding.kv_evict_paged(c.kp, None, c.wp, c.table, c.seq_lens, c.cap, 70)
        for b, L in enumerate([500, 90]):
            want = ol.evict(f64(c.w[b, 0, :L]), 70, 0, 1)
            assert (kept[b, 0].cpu().numpy() == want).all()
            assert torch.equal(c.rows_back(c.kp)[b, :70, 0], c.k[b, torch.from_numpy(want).cuda(), 0])


@pytest.mark.parametrize("in_place", [False, True])
def test_long_eviction(in_place):
    c = Cache(1, [70000, 40000], 70001, 2, 64, 32)
    numbers(c, 2, "zeros")
    before = c.k.clone(), c.w.clone()
    kept, _, moved = evict(c, 9000, 4, 100, None if in_place else 9000)
    for b, L in enumerate([70000, 40000]):
        for h in range(2):
            want = ol.evict(f64(before[1][b, h, :L]), 9000, 4, 100)
            assert (kept[b, h].cpu().numpy() == want).all()
            at = torch.from_numpy(want).cuda()
            assert torch.equal(moved[0][b, :9000, h], before[0][b, at, h])
            assert torch.equal(moved[2][b, h, :9000], before[1][b, h, at])


@pytest.mark.parametrize("int8", [False, True])
def test_decode_weights_eviction_decode(int8):
    """Steps of a program with a budget: write, attend, weigh, and cut down when the cache is over it."""
    B, Hq, Hkv, D, page, budget = 3, 8, 2, 128, 16, 200
    lens = [215, 150, 199]
    table = torch.arange(B * 16, device="cuda", dtype=torch.int32).view(B, 16).contiguous()
    shape = (B * 16, page, Hkv, D)
    dt = torch.int8 if int8 else torch.bfloat16
    pools = [torch.zeros(shape, device="cuda", dtype=dt) for _ in "kv"]
    scales = [torch.zeros(B * 16, Hkv, page, device="cuda") for _ in "kv"]
    wpool = torch.zeros(B * 16, Hkv, page, device="cuda")
    seq = lens_of(*lens)
    gen = torch.Generator(device="cuda").manual_seed(5)
    acc = [[np.zeros(0) for _ in range(Hkv)] for _ in range(B)]

    def write(n):
        k, v = randn(gen, B, n, Hkv, D), randn(gen, B, n, Hkv, D)
        if int8:
            binding.kv_write_int8_paged(k, v, *pools, *scales, table, seq, 256)
        else:
            binding.kv_write_paged(k, v, *pools, table, seq, 256)

    def rows(b, h, x, L):
        t = torch.arange(L, device="cuda")
        y = f64(pools[x][table[b].long()[t // page], t % page, h])
        return y * f64(scales[x][table[b].long()[t // page], h, t % page])[:, None] if int8 else y

    write(max(lens))
    for step in range(12):
        L = seq.tolist()
        q = randn(gen, B, 1, Hq, D)
        if int8:
            out = binding.decode_attn_int8_paged(q[:, 0].contiguous(), *pools, *scales, table, seq, 256)
            binding.kv_weights_int8_paged(q, pools[0], scales[0], wpool, table, seq, 256)
        else:
            out = binding.decode_attn_paged(q[:, 0].contiguous(), *pools, table, seq, 256)
            binding.kv_weights_paged(q, pools[0], wpool, table, seq, 256)
        for b in range(B):
            for h in range(Hkv):
                k = rows(b, h, 0, L[b])
                w = ol.weights(f64(q[b])[:, h * 4:h * 4 + 4], k[:, None], D ** -0.5)[0]
                if step == 0 or len(acc[b][h]) != L[b]:
                    acc[b][h] = np.concatenate((acc[b][h], np.zeros(L[b] - len(acc[b][h]))))
                acc[b][h] += w
                t = torch.arange(L[b], device="cuda")
                got = f64(wpool[table[b].long()[t // page], h, t % page])
                e = score_error(f64(q[b]), k, D ** -0.5, D)
                assert (np.abs(got - acc[b][h]) <= w * (2 * e + 64 * 2.0 ** -24) + 2.0 ** -22 * acc[b][h]).all()
                acc[b][h] = got
                want, mass = ol.attend(f64(q[b])[:, h * 4:h * 4 + 4], k[:, None], rows(b, h, 1, L[b])[:, None], D ** -0.5)
                # decode of int8 rounds the weights to f16, of bf16 to bf16
                check_attention(f64(out[b:b + 1, h * 4:h * 4 + 4]), want, mass, score_error(f64(q[b]), k, D ** -0.5, D))
        if max(L) > budget:
            args = (*pools, *scales, wpool) if int8 else (*pools, wpool)
            fn = binding.kv_evict_int8_paged if int8 else binding.kv_evict_paged
            kept, new_lens = fn(*args, table, seq, 256, budget - 20, first=4, recent=32)
            for b in range(B):
                for h in range(Hkv):
                    want = ol.evict(acc[b][h], budget - 20, 4, 32)
                    assert (kept[b, h, :len(want)].cpu().numpy() == want).all()
                    acc[b][h] = acc[b][h][want]
            seq.copy_(new_lens)
        seq += 1
        write(1)
    assert binding.device_error() == 0


def test_captured_and_replayed():
    c = Cache(11, [900, 800], 1000, 2, 128, 16)
    numbers(c, 3, "plain")
    q, ws = randn(c.gen, 2, 1, 8, 128), binding.weights_workspace(2, 1, 8, 2, c.cap)
    out = c.wp.clone()
    to = dict(kept=torch.empty(2, 2, 100, device="cuda", dtype=torch.int32), new_lens=lens_of(0, 0),
              k_out=torch.zeros(2, 100, 2, 128, device="cuda", dtype=torch.bfloat16),
              v_out=torch.zeros(2, 100, 2, 128, device="cuda", dtype=torch.bfloat16),
              weights_out=torch.zeros(2, 2, 100, device="cuda"))

    def step():
        binding.kv_weights_paged(q, c.kp, c.wp, c.table, c.seq_lens, c.cap, workspace=ws, out=out)
        binding.kv_evict_paged(c.kp, c.vp, out, c.table, c.seq_lens, c.cap, 100, first=2, recent=8, **to)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for cut in (0, 300, 750):
        c.seq_lens.copy_(lens_of(900 - cut, 800))
        q.copy_(torch.randn(q.shape, device="cuda", generator=c.gen))
        ws.fill_(0xFF)
        graph.replay()
        got = [t.clone() for t in (out, *to.values())]
        step()
        assert all(torch.equal(a.view(torch.int32) if a.dtype == torch.float32 else a,
                               b.view(torch.int32) if b.dtype == torch.float32 else b) for a, b in zip(got, (out, *to.values())))


def test_bad_pages_are_flagged():
    c = Cache(12, [90, 80], 96, 2, 64, 16)
    numbers(c, 1, "plain")
    q = randn(c.gen, 2, 1, 4, 64)
    c.table[0, 2] = 10 ** 6
    c.kp, c.wp = c.kp.nan_to_num(), c.wp.nan_to_num()
    before = c.wp.clone()
    weigh(c, q, c.wp)
    assert binding.device_error() == 4
    kept, _ = binding.kv_evict_paged(c.kp, c.vp, c.wp, c.table, c.seq_lens, c.cap, 40)
    assert binding.device_error() == 4
    assert before.shape == c.wp.shape


def test_refusals():
    c = Cache(13, [90, 80], 96, 2, 64)
    numbers(c, 1, "plain")
    q = randn(c.gen, 2, 1, 4, 64)
    ok = (c.k, c.v, c.w, c.seq_lens)
    for keep, first, recent in ((8, 5, 4), (8, -1, 1), (8, 0, -1)):
        with pytest.raises(binding.DecodeAttnError):
            binding.kv_evict_contig(*ok, keep, first=first, recent=recent)
    with pytest.raises(ValueError, match="keep"):
        binding.kv_evict_contig(*ok, 0)
    with pytest.raises(ValueError, match="room"):
        binding.kv_evict_contig(*ok, 8, k_out=c.k[:, :4].contiguous(), v_out=c.v[:, :4].contiguous())
    with pytest.raises(binding.DecodeAttnError):  # the output is the cache
        binding.kv_evict_contig(*ok, 8, k_out=c.k, v_out=c.v)
    with pytest.raises(binding.DecodeAttnError):
        binding.kv_evict_contig(c.k, c.k, c.w, c.seq_lens, 8)
    with pytest.raises(ValueError, match="k_out"):
        binding.kv_evict_contig(*ok, 8, weights_out=c.w.clone())
    with pytest.raises(binding.DecodeAttnError):
        weigh(c, q, c.w, decay=float("inf"))
    with pytest.raises(binding.DecodeAttnError):  # more rows than are built
        weigh(c, randn(c.gen, 2, 600, 4, 64), c.w)
    with pytest.raises(binding.DecodeAttnError):
        weigh(c, q, c.w, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError, match="out"):
        weigh(c, q, c.w, out=c.w[:, :1])
    torch.cuda.synchronize()
    assert binding.device_error() == 0
