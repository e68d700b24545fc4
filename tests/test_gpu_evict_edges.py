"""Eviction and weights at their edges: pages outside the pool, and caches without a token."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from long_cache_helpers import Cache, f64, lens_of, randn, score_error  # noqa: E402
from oracle import long_cache as ol  # noqa: E402
from gqa_split_kv_gb300 import binding  # noqa: E402


def with_bad_page(int8, names, column=2):
    """Two sequences of 90 and 80 tokens in pages of 16; the first one's page of tokens 32 .. 47 lies outside the pool.
    Every cell of the pools is finite.  Returns the cache and the page that it had."""
    c = Cache(12, [90, 80], 96, 2, 64, 16, names=names, int8=int8)
    c.put_numbers("w", torch.rand(2, 2, 96, generator=c.gen, device="cuda"))
    for x in ("kp", "vp", "ksp", "vsp", "wp"):
        if hasattr(c, x) and getattr(c, x).is_floating_point():
            getattr(c, x).nan_to_num_(7.0)
    lost = int(c.table[0, column])
    c.table[0, column] = 10 ** 6
    return c, lost


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("n", [1, 3, 40])
def test_weights_do_not_write_for_a_page_outside_the_pool(int8, n):
    c, lost = with_bad_page(int8, "k")
    q = randn(c.gen, 2, n, 4, 64)
    before = c.wp.clone()
    if int8:
        binding.kv_weights_int8_paged(q, c.kp, c.ksp, c.wp, c.table, c.seq_lens, c.cap)
    else:
        binding.kv_weights_paged(q, c.kp, c.wp, c.table, c.seq_lens, c.cap)
    assert binding.device_error() == 4
    live = torch.zeros_like(c.wp, dtype=torch.bool)
    for b, t0, t1, page in c.places():
        if page != 10 ** 6:
            live[page, :, :t1 - t0] = True
    assert not live[lost].any()
    assert torch.equal(c.wp[~live], before[~live])
    assert (c.wp[live] >= before[live]).all()
    k = c.values("k", 1)  # the other sequence is what it is without the bad page
    w = ol.weights(f64(q[1]), k, 0.125)
    tol = w * (2 * score_error(f64(q[1]), k, 0.125, 64) + (2 * n + 64) * 2.0 ** -24)
    for t0 in range(0, 80, 16):
        page = int(c.table[1, t0 // 16])
        got = f64(c.wp[page]) - f64(before[page])
        assert (np.abs(got - w[:, t0:t0 + 16]) <= tol[:, t0:t0 + 16] + 2.0 ** -23 * (w[:, t0:t0 + 16] + 1)).all()


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("column", [0, 2, 4])
def test_eviction_with_a_page_outside_the_pool(int8, in_place, column):
    """Rows from it are zeros, rows to it are not written, and the other sequence is cut as ever."""
    keep, first, recent = 40, 2, 8
    c, lost = with_bad_page(int8, "kv", column)
    names = ("k", "v", "ks", "vs", "w") if int8 else ("k", "v", "w")
    pools = [getattr(c, x + "p") for x in names]
    before = [p.clone() for p in pools]
    out = {}
    if not in_place:
        out = dict(k_out=torch.full((2, keep, 2, 64), 3, device="cuda").to(c.k.dtype))
        out["v_out"] = out["k_out"].clone()
        if int8:
            out["k_scale_out"], out["v_scale_out"] = (torch.full((2, 2, keep), 5.0, device="cuda") for _ in "kv")
        out["weights_out"] = torch.full((2, 2, keep), 5.0, device="cuda")
    fn = binding.kv_evict_int8_paged if int8 else binding.kv_evict_paged
    kept, new_lens = fn(*pools, c.table, c.seq_lens, c.cap, keep, first=first, recent=recent, **out)
    assert binding.device_error() == 4
    assert new_lens.tolist() == [keep, keep]
    bad = 10 ** 6
    place = lambda b, t: (int(c.table[b, t // 16]), t % 16)  # noqa: E731
    want = [p.clone() for p in before]  # in place: what each pool has to hold
    for b, L in enumerate((90, 80)):
        for h in range(2):
            at = kept[b, h].cpu().numpy()
            assert (np.diff(at) > 0).all() and at[0] >= 0 and at[-1] == L - 1
            if b == 1:
                w = [float(before[-1][place(1, t)[0], h, place(1, t)[1]]) for t in range(L)]
                assert (at == ol.evict(np.array(w), keep, first, recent)).all()
            for x, p in enumerate(before):
                cell = lambda q, page, row: q[page, row, h] if q.dim() == 4 else q[page, h, row]  # noqa: E731
                for i, t in enumerate(at):
                    page, row = place(b, int(t))
                    value = torch.zeros_like(cell(p, 0, 0)) if page == bad else cell(p, page, row)
                    if not in_place:
                        y = list(out.values())[x]
                        assert torch.equal(y[b, i, h] if y.dim() == 4 else y[b, h, i], value), (b, h, x, i, t)
                    elif place(b, i)[0] != bad and t != i:
                        cell(want[x], *place(b, i)).copy_(value)
                if in_place and x == len(before) - 1:
                    for t in range(keep, L):
                        if place(b, t)[0] != bad:
                            cell(want[x], *place(b, t)).zero_()
    for p, y in zip(pools, want if in_place else before):
        assert torch.equal(p, y)


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("int8", [False, True])
def test_a_cache_without_a_token(paged, int8):
    """Rows and pages that do not exist: nothing is kept, and the weights of the outputs are zeros."""
    dt = torch.int8 if int8 else torch.bfloat16
    slabs, slab = (0, 16) if paged else (2, 0)
    k, v = (torch.empty(slabs, slab, 3, 32, dtype=dt, device="cuda") for _ in "kv")
    numbers = [torch.empty(slabs, 3, slab, device="cuda") for _ in range(3 if int8 else 1)]
    out = dict(k_out=torch.full((2, 6, 3, 32), 3, device="cuda").to(dt), weights_out=torch.full((2, 3, 6), 5.0, device="cuda"))
    out["v_out"] = out["k_out"].clone()
    if int8:
        out["k_scale_out"], out["v_scale_out"] = (torch.full((2, 3, 6), 5.0, device="cuda") for _ in "kv")
    old = {x: y.clone() for x, y in out.items()}
    pages = (torch.zeros(2, 4, dtype=torch.int32, device="cuda"), lens_of(5, 0), 64) if paged else (lens_of(5, 0),)
    fn = getattr(binding, "kv_evict" + ("_int8" if int8 else "") + ("_paged" if paged else "_contig"))
    kept, new_lens = fn(k, v, *numbers, *pages, 4, **out)
    assert (kept == -1).all() and new_lens.tolist() == [0, 0]
    assert not out["weights_out"].any()
    for x in out:
        if x != "weights_out":
            assert torch.equal(out[x], old[x])
    assert binding.device_error() == 0


@pytest.mark.parametrize("B,L,keep", [(1, 500_000, 300_000), (1, 500_000, 700), (330, 50_000, 900)])
def test_more_weights_than_shared_memory_holds(B, L, keep):
    """One sequence whose share of a cluster's CTA is more than its shared memory, and many of a CTA each."""
    gen = torch.Generator(device="cuda").manual_seed(L)
    k = torch.arange(L, device="cuda", dtype=torch.int32).view(1, L, 1, 1).expand(B, L, 1, 4).contiguous().view(torch.bfloat16)
    w = (torch.rand(B, 1, L, generator=gen, device="cuda") * 5000).floor()  # with ties
    before = w.clone()
    kept, new_lens = binding.kv_evict_contig(k, None, w, None, keep, first=3, recent=50)
    assert new_lens.tolist() == [keep] * B
    for b in sorted({0, B // 2, B - 1}):
        want = ol.evict(f64(before[b, 0]), keep, 3, 50)
        assert (kept[b, 0].cpu().numpy() == want).all()
        at = torch.from_numpy(want).cuda()
        assert torch.equal(k[b, :keep, 0].view(torch.int32), at.to(torch.int32)[:, None].expand(keep, 4))
        assert torch.equal(w[b, 0, :keep], before[b, 0, at]) and not w[b, 0, keep:].any()
    assert binding.device_error() == 0
