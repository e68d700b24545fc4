"""GPU parity of attention behind a shared prefix against the CPU oracle, and the ways it is used."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from long_cache_helpers import Cache, check_attention, f64, lens_of, randn, score_error  # noqa: E402
from oracle import long_cache as ol  # noqa: E402
from gqa_split_kv_gb300 import binding  # noqa: E402


class Shared:
    """A batch behind a prefix of P tokens: lens count it."""

    def __init__(self, seed, P, lens, n, Hq, Hkv, D, page=0, rest=None):
        self.P, self.n, self.Hq, self.D, self.page = P, n, Hq, D, page
        rest = max([max(L - P, 0) for L in lens] + [1]) + 3 if rest is None else rest
        self.lens = lens
        gen = torch.Generator(device="cuda").manual_seed(seed + 1)
        self.q = randn(gen, len(lens), n, Hq, D)
        self.kp, self.vp = randn(gen, P, Hkv, D), randn(gen, P, Hkv, D)
        self.seq_lens = lens_of(*lens)
        if page:
            # every sequence's tokens from its last shared page's start on are its own pages
            start = P // page * page
            c = Cache(seed, [max(L - start, 0) for L in lens], rest + P - start, Hkv, D, page)
            c.cap_total = start + c.cap
            last = -(-P // page)
            pages = torch.arange(last, device="cuda", dtype=torch.int32)
            c.table = torch.where(c.table >= 0, c.table + last, c.table)
            bad = torch.full((len(lens), P // page), 1 << 30, dtype=torch.int32, device="cuda")  # never read
            self.table = torch.cat((bad, c.table), 1).contiguous()
            self.prefix_table = pages.flip(0).contiguous()
            for x, head in (("k", self.kp), ("v", self.vp)):
                own = torch.full((last, page, Hkv, D), float("nan"), dtype=torch.bfloat16, device="cuda")
                for j in range(last):
                    t1 = min(P, (j + 1) * page)
                    own[int(self.prefix_table[j]), :t1 - j * page] = head[j * page:t1]
                setattr(self, x + "_pool", torch.cat((own, getattr(c, x + "p"))))
            self.own_start, self.max_len = start, c.cap_total
        else:
            c = Cache(seed, [max(L - P, 0) for L in lens], rest, Hkv, D)
            self.own_start = P
        self.c = c

    def run(self, **kw):
        if self.page:
            return binding.prefix_attn_paged(self.q, self.k_pool, self.v_pool, self.prefix_table, self.P, self.table,
                                             self.seq_lens, self.max_len, **kw)
        return binding.prefix_attn_contig(self.q, self.kp, self.vp, self.c.k, self.c.v, self.seq_lens, **kw)

    def check(self, out, scale=None):
        scale = self.D ** -0.5 if scale is None else scale
        out = f64(out)
        for b, L in enumerate(self.lens):
            k, v = (np.concatenate((f64(head)[:max(L, 0)], own[max(self.P - self.own_start, 0):])) if L > self.P else
                    f64(head)[:max(L, 0)] for head, own in ((self.kp, self.c.values("k", b)), (self.vp, self.c.values("v", b))))
            q = f64(self.q[b])
            want, mass = ol.attend(q, k, v, scale)
            check_attention(out[b], want, mass, score_error(q, k, scale, self.D))


@pytest.mark.parametrize("page", [0, 16, 48])
@pytest.mark.parametrize("D,Hq,Hkv", [(64, 6, 2), (128, 8, 2), (128, 5, 5), (256, 6, 1), (128, 64, 1)])
@pytest.mark.parametrize("P,lens,n", [
    (100, [101, 130, 100 + 64, 100 + 65, 100 + 200], 1),
    (1, [2, 1, 0, 70], 1),
    (257, [300, 257, 256, 100, 0, 3, 258], 3),
    (64, [64 + 16, 64 + 17, 500, 64], 16),
    (1000, [1001], 1),
])
def test_against_the_oracle(page, D, Hq, Hkv, P, lens, n):
    s = Shared(P + D + n, P, lens, n, Hq, Hkv, D, page)
    out = torch.full_like(s.q, float("nan"))
    assert s.run(out=out) is out
    s.check(out)
    assert binding.device_error() == 0


@pytest.mark.parametrize("page", [0, 32])
@pytest.mark.parametrize("B,n,Hq,Hkv,D,P", [(40, 1, 16, 2, 128, 700), (9, 5, 24, 4, 256, 333), (3, 200, 4, 2, 64, 129),
                                            (70, 4, 8, 1, 128, 2100), (33, 16, 8, 2, 256, 500)])
def test_many_rows(page, B, n, Hq, Hkv, D, P):
    rng = np.random.default_rng(B)
    lens = [P + n + int(x) for x in rng.integers(0, 90, B)]
    lens[B // 2] = 0
    s = Shared(B, P, lens, n, Hq, Hkv, D, page)
    s.check(s.run())
    assert binding.device_error() == 0


@pytest.mark.parametrize("page", [0, 48])
@pytest.mark.parametrize("B,n,Hq,Hkv,D,P", [(8, 1, 64, 8, 128, 2300), (8, 1, 24, 4, 256, 2300), (3, 5, 8, 2, 64, 5000),
                                            (8, 1, 32, 8, 128, 300), (5, 3, 8, 2, 256, 130), (3, 5, 16, 4, 64, 512)])
def test_short_rests(page, B, n, Hq, Hkv, D, P):
    """Prefixes that share the card with their rests, and ones that few rows read like rests."""
    lens = [P + n + 9 * b for b in range(B)]
    lens[-1], lens[0] = P // 2, P
    s = Shared(B, P, lens, n, Hq, Hkv, D, page)
    s.check(s.run())
    assert binding.device_error() == 0


@pytest.mark.parametrize("n,Hq,Hkv,D", [(1, 8, 2, 128), (5, 24, 2, 256), (9, 8, 1, 64), (9, 16, 1, 128)])
def test_growing_scores(n, Hq, Hkv, D):
    """Scores that grow along the prefix and the rests: running maxima are raised again and again."""
    P = 1500
    s = Shared(D, P, [P + 300, P + 20, P, 700, 0], n, Hq, Hkv, D, rest=300)
    s.kp.mul_(torch.linspace(0.1, 9, P, device="cuda").view(P, 1, 1))
    s.c.k.mul_(torch.linspace(9, 12, 300, device="cuda").view(1, 300, 1, 1))
    s.check(s.run())


@pytest.mark.parametrize("scale", [0.0, -0.3, 2.0])
def test_scales(scale):
    s = Shared(5, 90, [91, 140], 1, 8, 2, 128)
    s.check(s.run(scale=scale), scale)


@pytest.mark.parametrize("D,Hq,Hkv", [(64, 8, 4), (128, 8, 2), (256, 12, 2), (128, 20, 1)])
@pytest.mark.parametrize("B", [1, 9])
def test_values_that_a_row_does_not_see_do_not_reach_it(D, Hq, Hkv, B):
    """Infinities and NaN in the keys and values of new tokens: only the tokens from them on are touched."""
    n, P = 5, 70
    lens = [P + 3 + 17 * b + n for b in range(B)]
    s = Shared(D + B, P, lens, n, Hq, Hkv, D)
    clean = s.run()
    for x, bad in ((s.c.v, float("inf")), (s.c.v, float("nan")), (s.c.k, float("nan"))):
        keep = x.clone()
        for b, L in enumerate(lens):
            x[b, L - P - 2, :, 3:9] = bad  # the last token but one
        out = s.run()
        assert torch.equal(out[:, :n - 2], clean[:, :n - 2])
        assert not torch.isfinite(out[:, n - 2:]).all(-1).any()
        x.copy_(keep)


def test_no_prefix_and_no_rest():
    s = Shared(6, 0, [5, 300], 2, 4, 2, 64)
    s.check(s.run())
    s = Shared(7, 500, [500, 480, 500], 2, 4, 2, 64)
    s.check(s.run())
    s = Shared(7, 500, [500, 480, 500], 2, 4, 2, 64, page=16)
    s.check(s.run())


def test_null_lengths_are_the_capacity():
    s = Shared(8, 77, [77 + 40] * 3, 2, 8, 2, 128, rest=40)
    want = s.run()
    got = binding.prefix_attn_contig(s.q, s.kp, s.vp, s.c.k, s.c.v)
    assert torch.equal(got, want)
    s.seq_lens = lens_of(10 ** 9, 2 ** 31 - 1, 77 + 40)  # clamped
    assert torch.equal(s.run(), want)
    s.seq_lens = lens_of(-5, 117, -2 ** 31)
    got = s.run()
    assert torch.equal(got[1], want[1]) and not got[0].any() and not got[2].any()


def test_equals_decode_over_the_whole_sequences():
    """The same tokens as ordinary sequences: both within a bf16 step of each other's sums."""
    s = Shared(9, 640, [641, 800, 1000], 1, 16, 4, 128)
    k, v = (torch.cat((p[None].expand(3, -1, -1, -1), own), 1).contiguous() for p, own in ((s.kp, s.c.k), (s.vp, s.c.v)))
    k, v = k.nan_to_num(), v.nan_to_num()
    want = binding.decode_attn_contig(s.q[:, 0].contiguous(), k, v, s.seq_lens)
    assert (s.run()[:, 0].float() - want.float()).abs().max() <= 2 * 2.0 ** -8 * 4


def test_bad_pages_are_flagged():
    s = Shared(10, 64, [100, 90], 1, 4, 2, 64, page=16)
    s.k_pool, s.v_pool = s.k_pool.nan_to_num(), s.v_pool.nan_to_num()
    s.table[0, 4] = 10 ** 6
    s.prefix_table[1] = -3
    out = s.run()
    assert torch.isfinite(out).all()
    assert binding.device_error() == 4
    assert binding.device_error() == 0


@pytest.mark.parametrize("P,lens", [(300, [310, 350, 400]), (3000, [3001] * 40)])
def test_captured_with_new_lengths_and_tokens(P, lens):
    s = Shared(11, P, lens, 1, 16, 2, 128, page=16)
    out, ws = torch.empty_like(s.q), binding.prefix_workspace(len(lens), 1, 16, 2, 128)
    s.run(out=out, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.run(out=out, workspace=ws)
    for cut in (0, 7, 9):
        s.lens = [max(L - cut * (i % 2), 0) for i, L in enumerate(lens)]
        s.seq_lens.copy_(lens_of(*s.lens))
        s.q.copy_(torch.randn(s.q.shape, device="cuda", generator=torch.Generator("cuda").manual_seed(cut)))
        ws.fill_(0xFF)  # nothing is kept in it
        graph.replay()
        got = out.clone()
        assert torch.equal(got, s.run())
        s.c.live = [max(L - s.own_start, 0) for L in s.lens]
        s.check(got)


def test_another_stream_and_repeats_are_bitwise_the_same():
    s = Shared(12, 1500, [1501 + 13 * i for i in range(20)], 2, 32, 8, 128)
    want = s.run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = [s.run(stream=side) for _ in range(3)]
    side.synchronize()
    assert all(torch.equal(g, want) for g in got)


def test_refusals():
    s = Shared(13, 100, [110, 120], 1, 8, 2, 128, page=16)
    for bad in (dict(out=s.q), dict(workspace=torch.empty(16, dtype=torch.uint8, device="cuda")), dict(scale=float("nan"))):
        with pytest.raises(binding.DecodeAttnError):
            s.run(**bad)
    with pytest.raises(ValueError, match="prefix_table"):
        binding.prefix_attn_paged(s.q, s.k_pool, s.v_pool, s.prefix_table[:3].contiguous(), 100, s.table, s.seq_lens, 200)
    with pytest.raises(ValueError, match="k_prefix"):
        binding.prefix_attn_contig(s.q, s.kp.float(), s.vp, s.c.k, s.c.v)
    with pytest.raises(binding.DecodeAttnError):  # a head's width that is not built
        q = torch.zeros(1, 1, 4, 96, device="cuda", dtype=torch.bfloat16)
        binding.prefix_attn_contig(q, q[0].expand(8, 4, 96).contiguous(), q[0].expand(8, 4, 96).contiguous(), q, q)
    with pytest.raises(ValueError, match="gradient"):
        binding.prefix_attn_contig(s.q, s.kp, s.vp, s.c.k, s.c.v, out=s.q.float().to(torch.bfloat16).requires_grad_())
    torch.cuda.synchronize()
    assert binding.device_error() == 0
