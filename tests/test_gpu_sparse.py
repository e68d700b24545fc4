"""GPU parity of mean keys, block selection and attention over selected blocks against the CPU oracle."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from long_cache_helpers import Cache, check_attention, f64, lens_of, randn, score_error  # noqa: E402
from oracle import long_cache as ol  # noqa: E402
from gqa_split_kv_gb300 import binding  # noqa: E402


def means_of(c, block, n=None, out=None):
    if c.page:
        return binding.block_means_paged(c.kp, c.table, c.seq_lens, c.cap, block, n, out=out)
    return binding.block_means_contig(c.k, c.seq_lens, block, n, out=out)


@pytest.mark.parametrize("page", [0, 16, 48])
@pytest.mark.parametrize("D,Hkv", [(64, 1), (128, 8), (256, 3), (8, 2), (192, 16)])
@pytest.mark.parametrize("lens,n,block", [([0, 1, 63, 64, 65, 200], 1, 64), ([0, 5, 300, 299], 40, 16), ([700, 33], None, 128),
                                          ([70, 500], 0, 32), ([257, 256, 100], 1000, 24)])
def test_means(page, D, Hkv, lens, n, block):
    c = Cache(D + block, lens, max(lens) + 5, Hkv, D, page, names="k")
    blocks = -(-c.cap // block) + 1
    out = torch.full((c.B, Hkv, blocks, D), 7.0, device="cuda", dtype=torch.bfloat16)
    assert means_of(c, block, n, out) is out
    got = f64(out)
    for b, L in enumerate(lens):
        k = c.values("k", b)
        want = ol.block_means(k, block, c.cap if n is None else n)
        for j in range(blocks):
            if j not in want:
                assert (got[b, :, j] == 7).all()
                continue
            # a sum of `block` terms in fp32, a division, one rounding to bf16
            tol = 2.0 ** -8 * np.abs(want[j]) + (block + 2) * 2.0 ** -24 * np.abs(k[j * block:(j + 1) * block]).mean(0)
            assert (np.abs(got[b, :, j] - want[j]) <= tol).all()
    made = means_of(c, block, n)
    assert torch.equal(made[:, :, :blocks - 1], torch.where(out == 7, 0, out)[:, :, :made.shape[2]])


def make_select(seed, B, n, Hq, Hkv, D, blocks):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return randn(gen, B, n, Hq, D), randn(gen, B, Hkv, blocks, D)


def check_select(q, means, lens, block, pick, first, recent):
    got = binding.block_select(q, means, lens_of(*lens), block, pick, first=first, recent=recent).cpu().numpy()
    cap = means.shape[2] * block
    for b, L in enumerate(lens):
        want = ol.select(f64(q[b]), f64(means[b]), min(max(L, 0), cap), block, pick, first, recent)
        assert (got[b] == want).all(), (b, L)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("Hq,Hkv", [(8, 2), (6, 1), (40, 2), (3, 3), (64, 1)])
@pytest.mark.parametrize("lens,n,block,pick,first,recent", [
    ([0, 1, 64, 65, 1000, 2047], 1, 64, 8, 1, 1),
    ([2000, 3, 1999], 5, 16, 30, 0, 1),
    ([500, 0, 40], 60, 32, 4, 2, 2),
    ([10 ** 9, 777], 2, 16, 1, 0, 1),
    ([2048], 1, 16, 200, 3, 9),
])
def test_selection(D, Hq, Hkv, lens, n, block, pick, first, recent):
    q, means = make_select(D + n, len(lens), n, Hq, Hkv, D, 2048 // block)
    check_select(q, means, lens, block, pick, first, recent)


@pytest.mark.parametrize("blocks,pick", [(1024, 64), (8192, 100), (3001, 2999)])
def test_long_selection(blocks, pick):
    q, means = make_select(blocks, 2, 1, 16, 2, 128, blocks)
    check_select(q, means, [blocks * 16, blocks * 16 - 40], 16, pick, 1, 2)


@pytest.mark.parametrize("n", [1, 7])
def test_selection_with_ties_and_special_scores(n):
    """Equal scores go to the lower block; scores closer than fp32 sums can tell are told apart; NaN is lowest."""
    D, blocks = 128, 200
    q, means = make_select(n, 4, n, 4, 2, D, blocks)
    q[0] = 0  # every score ties
    means[1, :, 10:150] = means[1, :, 10:11]  # most tie
    # neighbours that differ by 2^-24 of their terms: an fp32 sum loses that
    means[2] = 0
    means[2, ..., 0] = 1.0
    means[2, ..., 1] = -1.0
    q[2, ..., 0] = q[2, ..., 1] = 4096.0
    q[2, ..., 2:] = 0
    q[2, ..., 2] = 2.0 ** -12
    means[2, :, :, 2] = torch.randperm(blocks, device="cuda").to(torch.bfloat16) / 256
    means[3, :, 30:60, 5] = float("nan")
    means[3, :, 70, 9] = float("inf")
    lens = [blocks * 32] * 4
    check_select(q, means, lens, 32, 50, 1, 1)
    check_select(q, means, lens, 32, 1, 0, 1)


def listed(c, q, blocks, block, scale=None, **kw):
    if c.page:
        return binding.sparse_attn_paged(q, c.kp, c.vp, blocks, c.table, c.seq_lens, c.cap, block, scale=scale, **kw)
    return binding.sparse_attn_contig(q, c.k, c.v, blocks, c.seq_lens, block, scale=scale, **kw)


def check_sparse(c, q, blocks, block, out, scale=None):
    D = q.shape[-1]
    scale = D ** -0.5 if scale is None else scale
    got, host = f64(out), blocks.cpu().numpy()
    for b in range(c.B):
        k, v = c.values("k", b), c.values("v", b)
        tokens = [[ol.block_tokens(host[b, i, h], block) for h in range(c.H)] for i in range(q.shape[1])]
        want, mass = ol.attend(f64(q[b]), k, v, scale, tokens)
        check_attention(got[b], want, mass, score_error(f64(q[b]), k, scale, D))


@pytest.mark.parametrize("page", [0, 16, 48])
@pytest.mark.parametrize("D,Hq,Hkv", [(64, 8, 4), (128, 8, 2), (256, 6, 1), (128, 40, 1), (128, 3, 3)])
@pytest.mark.parametrize("lens,n,block,pick", [([0, 1, 64, 100, 700], 1, 64, 4), ([333, 50], 9, 16, 7), ([500, 2], 2, 48, 1),
                                               ([600, 600, 601], 1, 128, 5)])
def test_listed_blocks(page, D, Hq, Hkv, lens, n, block, pick):
    c = Cache(D + n, lens, max(lens) + 30, Hkv, D, page)
    q = randn(c.gen, c.B, n, Hq, D)
    rng = np.random.default_rng(pick)
    blocks = rng.integers(-2, max(lens) // block + 3, (c.B, n, Hkv, pick)).astype(np.int32)  # any order, some twice
    blocks[-1, 0, 0] = -1  # nothing at all
    blocks[0, 0, 0, 0] = 2 ** 31 - 1
    blocks = torch.from_numpy(blocks).cuda()
    out = torch.full_like(q, float("nan"))
    assert listed(c, q, blocks, block, out=out) is out
    check_sparse(c, q, blocks, block, out)
    assert binding.device_error() == 0


@pytest.mark.parametrize("page", [0, 32])
@pytest.mark.parametrize("B,n,Hq,Hkv,D,L,block,pick", [(1, 1, 32, 8, 128, 9000, 64, 32), (6, 1, 16, 2, 128, 5000, 64, 40),
                                                       (2, 70, 12, 2, 256, 1500, 32, 12), (1, 300, 4, 1, 64, 800, 16, 9)])
def test_a_step_means_selection_attention(page, B, n, Hq, Hkv, D, L, block, pick):
    """Keys written with their rotation, their blocks' means, the selection, the attention: as a program runs them."""
    lens = [L - 37 * b for b in range(B)]
    c = Cache(L + B, lens, L + 64, Hkv, D, page)
    q, new = randn(c.gen, B, n, Hq, D), randn(c.gen, B, n, Hkv, D)
    w = binding.rope_inv_freq(D)
    means = means_of(c, block)
    if page:
        binding.kv_write_paged(new, new, c.kp, c.vp, c.table, c.seq_lens, c.cap, inv_freq=w)
        c.k, c.v = (torch.where(torch.isnan(old), old, c.rows_back(p)) for old, p in ((c.k, c.kp), (c.v, c.vp)))
    else:
        binding.kv_write_contig(new, new, c.k, c.v, c.seq_lens, inv_freq=w)
    assert means_of(c, block, n, means) is means
    again = means_of(c, block)
    assert torch.equal(means, again)
    blocks = binding.block_select(q, means, c.seq_lens, block, pick)
    for b in range(B):
        assert (blocks[b].cpu().numpy() == ol.select(f64(q[b]), f64(means[b]), lens[b], block, pick, 1, 1)).all()
    check_sparse(c, q, blocks, block, listed(c, q, blocks, block))
    assert binding.device_error() == 0


def test_all_blocks_equal_decode():
    c = Cache(3, [900, 333], 1000, 2, 128)
    q = randn(c.gen, 2, 1, 16, 128)
    blocks = torch.arange(16, device="cuda", dtype=torch.int32).expand(2, 1, 2, 16).contiguous()
    k, v = c.k.nan_to_num(), c.v.nan_to_num()
    want = binding.decode_attn_contig(q[:, 0].contiguous(), k, v, c.seq_lens)
    assert (listed(c, q, blocks, 64)[:, 0].float() - want.float()).abs().max() <= 2 * 2.0 ** -8 * 4


def test_captured_and_replayed():
    c = Cache(4, [3000, 2000, 2500], 3100, 2, 128, 16)
    q = randn(c.gen, 3, 1, 16, 128)
    means, out = means_of(c, 64), torch.empty_like(q)
    blocks = binding.block_select(q, means, c.seq_lens, 64, 12)

    def step():
        means_of(c, 64, 1, means)
        binding.block_select(q, means, c.seq_lens, 64, 12, out=blocks)
        listed(c, q, blocks, 64, out=out)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for cut in (1, 500, 0):
        c.seq_lens.copy_(lens_of(3000 - cut, 2000, 2500 - cut))
        q.copy_(torch.randn(q.shape, device="cuda", generator=c.gen))
        graph.replay()
        got = out.clone(), blocks.clone()
        step()
        assert torch.equal(got[0], out) and torch.equal(got[1], blocks)


def test_refusals():
    c = Cache(5, [100, 90], 128, 2, 128)
    q = randn(c.gen, 2, 1, 8, 128)
    blocks = torch.zeros(2, 1, 2, 2, device="cuda", dtype=torch.int32)
    means = means_of(c, 64)
    for block in (24, 0):
        with pytest.raises(binding.DecodeAttnError):
            listed(c, q, blocks, block)
    with pytest.raises(binding.DecodeAttnError):
        listed(c, q, blocks, 64, out=q)
    with pytest.raises(ValueError, match="blocks"):
        listed(c, q, blocks.long(), 64)
    with pytest.raises(binding.DecodeAttnError):  # the forced blocks alone are more
        binding.block_select(q, means, c.seq_lens, 64, 2, first=2, recent=1)
    with pytest.raises(binding.DecodeAttnError):
        binding.block_select(q, means, c.seq_lens, 64, 2, first=1, recent=0)
    with pytest.raises(binding.DecodeAttnError):  # no room for the cache's last blocks
        means_of(c, 64, 1, torch.zeros(2, 2, 1, 128, device="cuda", dtype=torch.bfloat16))
    torch.cuda.synchronize()
    assert binding.device_error() == 0
