"""Prefix attention, selected blocks, weights and eviction beyond their own tests: caches past 2^31 elements, batches
of many sequences, nothing to do, streams side by side, captured forks, and what autograd sees."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from long_cache_helpers import Cache, check_attention, f64, lens_of, randn, score_error  # noqa: E402
from oracle import long_cache as ol  # noqa: E402
from gqa_split_kv_gb300 import binding  # noqa: E402


@pytest.fixture
def far():
    """Pools of more than 2^31 elements (and 2^32 bytes), used at their end."""
    H, D, page, pages = 8, 128, 64, 33000
    assert pages * page * H * D > 2 ** 31
    gen = torch.Generator(device="cuda").manual_seed(1)
    pools = [torch.zeros(pages, page, H, D, device="cuda", dtype=torch.bfloat16) for _ in "kv"]
    table = torch.arange(pages - 12, pages, device="cuda", dtype=torch.int32).flip(0).view(2, 6).contiguous()
    lens = [300, 377]
    rows = [randn(gen, 2, 384, H, D) for _ in "kv"]
    for pool, r in zip(pools, rows):
        pool[table.long()] = r.view(2, 6, page, H, D)
    yield dict(pools=pools, table=table, lens=lens, rows=rows, H=H, D=D, page=page, gen=gen)
    torch.cuda.empty_cache()


def test_far_prefix_and_blocks(far):
    q = randn(far["gen"], 2, 1, 16, 128)
    lens = lens_of(*far["lens"])
    means = binding.block_means_paged(far["pools"][0], far["table"], lens, 384, 64)
    blocks = binding.block_select(q, means, lens, 64, 3)
    sparse = binding.sparse_attn_paged(q, *far["pools"], blocks, far["table"], lens, 384, 64)
    prefix = binding.prefix_attn_paged(q, *far["pools"], far["table"][0].contiguous(), 128, far["table"], lens, 384)
    host = blocks.cpu().numpy()
    for b, L in enumerate(far["lens"]):
        k, v = (f64(r[b, :L]) for r in far["rows"])
        e = score_error(f64(q[b]), k, 128 ** -0.5, 128)
        want = ol.block_means(k, 64, L)
        for j, m in want.items():
            assert np.abs(f64(means[b, :, j]) - m).max() <= 2.0 ** -8 * np.abs(m).max() + 2.0 ** -16
        assert (host[b] == ol.select(f64(q[b]), f64(means[b]), L, 64, 3, 1, 1)).all()
        out, mass = ol.attend(f64(q[b]), k, v, 128 ** -0.5, [[ol.block_tokens(host[b, 0, h], 64) for h in range(8)]])
        check_attention(f64(sparse[b]), out, mass, e)
        first = [f64(r[0, :128]) for r in far["rows"]]  # the prefix is sequence 0's
        out, mass = ol.attend(f64(q[b]), np.concatenate((first[0], k[128:])), np.concatenate((first[1], v[128:])), 128 ** -0.5)
        check_attention(f64(prefix[b]), out, mass, e)


def test_far_weights_and_eviction(far):
    q = randn(far["gen"], 2, 1, 16, 128)
    lens = lens_of(*far["lens"])
    pool = torch.zeros(far["pools"][0].shape[0], 8, 64, device="cuda")
    binding.kv_weights_paged(q, far["pools"][0], pool, far["table"], lens, 384)
    w = [ol.weights(f64(q[b]), f64(far["rows"][0][b, :L]), 128 ** -0.5) for b, L in enumerate(far["lens"])]
    got = pool[far["table"].long()].permute(0, 2, 1, 3).reshape(2, 8, 384)
    for b, L in enumerate(far["lens"]):
        assert np.abs(f64(got[b, :, :L]) - w[b]).max() <= 2.0 ** -10 and not got[b, :, L:].any()
    kept, new = binding.kv_evict_paged(*far["pools"], pool, far["table"], lens, 384, 100, first=2, recent=10)
    assert new.tolist() == [100, 100]
    for b, L in enumerate(far["lens"]):
        for h in range(8):
            want = ol.evict(f64(got[b, h, :L]), 100, 2, 10)
            assert (kept[b, h].cpu().numpy() == want).all()
            at = torch.from_numpy(want).cuda()
            t = torch.arange(100, device="cuda")
            for pl, r in zip(far["pools"], far["rows"]):
                assert torch.equal(pl[far["table"][b].long()[t // 64], t % 64, h], r[b, at, h])


@pytest.mark.parametrize("B", [513, 1500])
def test_batches_of_many_sequences(B):
    rng = np.random.default_rng(B)
    lens = rng.integers(0, 70, B).tolist()
    c = Cache(B, lens, 70, 1, 64)
    c.put_numbers("w", torch.zeros(B, 1, 70, device="cuda"))
    q = randn(c.gen, B, 1, 4, 64)
    kp, vp = randn(c.gen, 40, 1, 64), randn(c.gen, 40, 1, 64)
    out = binding.prefix_attn_contig(q, kp, vp, c.k, c.v, lens_of(*(40 + L if L else 0 for L in lens)))
    w = binding.kv_weights_contig(q, c.k, None, c.seq_lens)
    kept, new = binding.kv_evict_contig(c.k.clone(), c.v.clone(), w.clone(), c.seq_lens, 20, recent=4)
    assert new.tolist() == [min(L, 20) for L in lens]
    for b in list(range(0, B, 41)) + [B - 1]:
        L = lens[b]
        if L == 0:
            assert not out[b].any() and (kept[b] == -1).all()
            continue
        k, v = (np.concatenate((f64(p), c.values(x, b))) for p, x in ((kp, "k"), (vp, "v")))
        want, mass = ol.attend(f64(q[b]), k, v, 0.125)
        check_attention(f64(out[b]), want, mass, score_error(f64(q[b]), k, 0.125, 64))
        ws = ol.weights(f64(q[b]), c.values("k", b), 0.125)
        assert np.abs(f64(w[b, :, :L]) - ws).max() <= 2.0 ** -10
        assert (kept[b, 0, :min(L, 20)].cpu().numpy() == ol.evict(f64(w[b, 0, :L]), 20, 0, 4)).all()


def test_nothing_to_do():
    bf = dict(device="cuda", dtype=torch.bfloat16)
    q0, kv0 = torch.zeros(0, 1, 8, 128, **bf), torch.zeros(0, 64, 2, 128, **bf)
    none = torch.zeros(0, device="cuda", dtype=torch.int32)
    p = torch.ones(32, 2, 128, **bf)
    assert binding.prefix_attn_contig(q0, p, p, kv0, kv0, none).shape == q0.shape
    q, empty = torch.ones(3, 2, 8, 128, **bf), torch.zeros(3, 0, 2, 128, **bf)
    out = binding.prefix_attn_contig(q, p, p, empty, empty)  # every sequence the prefix alone
    assert torch.equal(out, torch.ones_like(out))
    assert not binding.prefix_attn_contig(q, p[:0], p[:0], empty, empty).any()
    pool, table = torch.zeros(0, 16, 2, 128, **bf), torch.zeros(3, 4, device="cuda", dtype=torch.int32)
    lens = lens_of(5, 0, 64)
    assert not binding.prefix_attn_paged(q, pool, pool, table[0].contiguous(), 20, table, lens, 64).any()
    blocks = torch.zeros(3, 2, 2, 4, device="cuda", dtype=torch.int32)
    assert not binding.sparse_attn_paged(q, pool, pool, blocks, table, lens, 64, 16).any()
    assert not binding.sparse_attn_contig(q, empty, empty, blocks, None, 16).any()
    assert binding.block_means_contig(empty, None, 16).shape == (3, 2, 0, 128)
    assert (binding.block_select(q, torch.zeros(3, 2, 0, 128, **bf), lens, 16, 4) == -1).all()
    w = binding.kv_weights_contig(torch.zeros(2, 0, 8, 128, **bf), torch.ones(2, 9, 2, 128, **bf),
                                  torch.full((2, 2, 9), 2.0, device="cuda"), decay=0.5)
    assert (w == 1).all()  # no new token: the decay alone
    kept, new = binding.kv_evict_contig(empty, empty, torch.zeros(3, 2, 0, device="cuda"), None, 5)
    assert (kept == -1).all() and not new.any()
    assert binding.kv_evict_paged(pool, pool, torch.zeros(0, 2, 16, device="cuda"), table, lens, 64, 5)[1].tolist() == [0, 0, 0]
    torch.cuda.synchronize()
    assert binding.device_error() == 0


def program(seed):
    """A program's steps on caches of its own, and what they leave."""
    c = Cache(seed, [700, 650, 90], 900, 2, 128, 16)
    c.put_numbers("w", torch.rand(3, 2, 900, generator=c.gen, device="cuda"))
    for x in ("kp", "vp", "wp"):
        setattr(c, x, getattr(c, x).nan_to_num())
    q, many = randn(c.gen, 3, 1, 16, 128), randn(c.gen, 3, 6, 16, 128)
    kpre, vpre = randn(c.gen, 333, 2, 128), randn(c.gen, 333, 2, 128)
    k, v = c.k.nan_to_num().contiguous(), c.v.nan_to_num().contiguous()
    lens = lens_of(333 + 700, 333 + 650, 0)
    means = binding.block_means_paged(c.kp, c.table, c.seq_lens, c.cap, 32)
    left = dict(prefix=torch.empty_like(many), sparse=torch.empty_like(q), blocks=torch.empty(3, 1, 2, 6, device="cuda", dtype=torch.int32),
                step=c.wp.clone(), window=c.wp.clone(), k=c.kp.clone(), v=c.vp.clone(), w=c.wp.clone(), means=means,
                kept=torch.empty(3, 2, 100, device="cuda", dtype=torch.int32), new=torch.empty(3, device="cuda", dtype=torch.int32))
    start = {x: left[x].clone() for x in ("k", "v", "w")}

    def step():
        for x in start:
            left[x].copy_(start[x])
        binding.prefix_attn_contig(many, kpre, vpre, k, v, lens, out=left["prefix"])
        binding.block_means_paged(c.kp, c.table, c.seq_lens, c.cap, 32, 1, out=left["means"])
        binding.block_select(q, left["means"], c.seq_lens, 32, 6, out=left["blocks"])
        binding.sparse_attn_paged(q, c.kp, c.vp, left["blocks"], c.table, c.seq_lens, c.cap, 32, out=left["sparse"])
        binding.kv_weights_paged(q, c.kp, c.wp, c.table, c.seq_lens, c.cap, out=left["step"])
        binding.kv_weights_paged(many, c.kp, c.wp, c.table, c.seq_lens, c.cap, out=left["window"])
        binding.kv_evict_paged(left["k"], left["v"], left["w"], c.table, c.seq_lens, c.cap, 100, first=3, recent=9,
                               kept=left["kept"], new_lens=left["new"])

    return step, left


def same(a, b):
    return all(torch.equal(a[x].view(torch.int8), b[x].view(torch.int8)) for x in a)


def test_two_programs_on_two_streams():
    (one, a), (two, b) = program(1), program(2)
    one(), two()
    torch.cuda.synchronize()
    want = [{x: t.clone() for x, t in d.items()} for d in (a, b)]
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(10):
        for s, f in zip(streams, (one, two)):
            with torch.cuda.stream(s):
                f()
    torch.cuda.synchronize()
    assert same(a, want[0]) and same(b, want[1])
    assert binding.device_error() == 0


def test_captured_fork():
    (one, a), (two, b) = program(3), program(4)
    one(), two()
    torch.cuda.synchronize()
    want = [{x: t.clone() for x, t in d.items()} for d in (a, b)]
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            two()
        one()
        torch.cuda.current_stream().wait_stream(side)
    for _ in range(5):
        for d in (a, b):
            for t in d.values():
                t.zero_() if t.dtype == torch.int32 else None
        graph.replay()
    torch.cuda.synchronize()
    assert same(a, want[0]) and same(b, want[1])
    assert binding.device_error() == 0


def test_outputs_count_as_changed_and_tracked_ones_are_refused():
    step, left = program(5)
    before = {x: t._version for x, t in left.items()}
    step()
    assert all(t._version > before[x] for x, t in left.items())
    w = torch.zeros(1, 2, 8, device="cuda", requires_grad=True)
    kv, q = torch.zeros(1, 8, 2, 64, device="cuda", dtype=torch.bfloat16), torch.zeros(1, 1, 2, 64, device="cuda", dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="gradient"):
        binding.kv_weights_contig(q, kv, w)
    with pytest.raises(ValueError, match="gradient"):
        binding.kv_evict_contig(kv, kv.clone(), w, None, 4)
    with torch.no_grad():
        binding.kv_weights_contig(q, kv, w)
    assert not binding.kv_weights_contig(q, kv, w.detach(), out=torch.zeros_like(w.detach())).requires_grad


def test_tensors_of_the_cpu_are_refused():
    q, kv = torch.zeros(1, 1, 2, 64, dtype=torch.bfloat16), torch.zeros(1, 8, 2, 64, dtype=torch.bfloat16)
    for call in (lambda: binding.prefix_attn_contig(q, kv[0], kv[0], kv, kv), lambda: binding.kv_weights_contig(q, kv, None),
                 lambda: binding.block_means_contig(kv), lambda: binding.block_select(q, kv[:, :2], None, 16, 2),
                 lambda: binding.kv_evict_contig(kv, kv, torch.zeros(1, 2, 8), None, 4)):
        with pytest.raises(ValueError):
            call()
