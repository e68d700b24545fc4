"""Attention weights where scores are not finite, where rows see different tokens, over lengths whose products pass 32 bits,
and with scales that differ from token to token."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from long_cache_helpers import Cache, f64, randn, score_error  # noqa: E402
from oracle import long_cache as ol  # noqa: E402
from gqa_split_kv_gb300 import binding  # noqa: E402


def weigh(c, q):
    if c.page:
        return c.numbers_back(binding.kv_weights_paged(q, c.kp, None, c.table, c.seq_lens, c.cap))
    return binding.kv_weights_contig(q, c.k, None, c.seq_lens)


def put(c, b, t, h, d, x):
    """Element d of token t's key becomes x, in the cache and in its pool."""
    c.k[b, t, h, d] = x
    if c.page:
        c.kp[int(c.table[b, t // c.page]), t % c.page, h, d] = x


def check(got, q, k, scale, finite):
    """The weights of one sequence; tolerance: twice a score's error, taken of the finite scores, and the sums'."""
    with np.errstate(invalid="ignore"):
        want = ol.weights(f64(q), k, scale)
    rows = q.shape[0] * q.shape[1] // k.shape[1]
    tol = want * (2 * score_error(f64(q), finite, scale, q.shape[-1]) + (rows + 64) * 2.0 ** -24) + rows * 1e-37
    got = f64(got)
    assert (np.isnan(got) == np.isnan(want)).all(), np.argwhere(np.isnan(got) != np.isnan(want))[:5]
    assert not (np.abs(got - want) > tol).any()
    return want


@pytest.mark.parametrize("page", [0, 16])
@pytest.mark.parametrize("D,rows", [(64, 3), (128, 13), (64, 17), (128, 33), (256, 40), (128, 96), (128, 145)])
def test_a_score_of_minus_infinity_is_a_weight_of_zero(D, rows, page):
    """An infinite key that every row scores -inf: its weight is 0 and the others' are what they are without it."""
    c = Cache(D + rows, [300, 77], 300, 2, D, page, names="k")
    q = randn(c.gen, 2, 1, 2 * rows if rows <= 64 else 2, D)
    if rows > 64:  # more rows than a group may have heads: several tokens
        q = randn(c.gen, 2, rows, 2, D)
    q[..., 5] = -q[..., 5].abs() - 0.5
    clean = [c.values("k", b) for b in range(2)]
    for b, t in ((0, 130), (1, 7)):
        for h in range(2):
            put(c, b, t, h, 5, float("inf"))
    got = weigh(c, q)
    for b, (L, t) in enumerate(((300, 130), (77, 7))):
        if q.shape[1] > L:  # (the first tokens see nothing)
            continue
        want = check(got[b, :, :L], q[b], c.values("k", b), D ** -0.5, clean[b])
        assert (want[:, t] == 0).all() and np.isfinite(want).all()
    assert binding.device_error() == 0


@pytest.mark.parametrize("page", [0, 32])
@pytest.mark.parametrize("n,G,D", [(2, 1, 64), (3, 4, 128), (5, 3, 256), (3, 8, 64), (7, 7, 128), (40, 4, 128), (20, 5, 256)])
def test_a_row_that_is_not_finite_reaches_the_tokens_it_sees(n, G, D, page):
    """The last token but one scores its own key +inf with one head, so that row is NaN; the last token's rows score that
    key -inf.  The last key is seen by the last token alone, and its weight is finite."""
    lens = [n + 90, 200]
    c = Cache(n + G + D, lens, 200, 2, D, page, names="k")
    q = randn(c.gen, 2, n, 2 * G, D)
    q[..., 5] = -q[..., 5].abs() - 0.5
    q[:, n - 2, ::G, 5] = 1.0
    clean = [c.values("k", b) for b in range(2)]
    for b, L in enumerate(lens):
        for h in range(2):
            put(c, b, L - 2, h, 5, float("inf"))
    got = weigh(c, q)
    for b, L in enumerate(lens):
        want = check(got[b, :, :L], q[b], c.values("k", b), D ** -0.5, clean[b])
        assert np.isnan(want[:, :L - 1]).all() and (want[:, L - 1] > 0).all()
    assert binding.device_error() == 0


def test_lengths_whose_products_with_the_group_pass_32_bits():
    """One new token of 64 heads over 34 million equal keys: every weight is 64 / L.  The sums of a CTA's range are whole
    numbers below 2^24, joining 304 of them rounds by 2^-24 each, and so do 64 additions and the reciprocal."""
    L, G, D = 34_000_000, 64, 64
    k = torch.zeros(1, L, 1, D, dtype=torch.int8, device="cuda")
    scale = torch.ones(1, 1, L, device="cuda")
    q = torch.randn(1, 1, G, D, device="cuda").to(torch.bfloat16)
    w = binding.kv_weights_int8_contig(q, k, scale, None)
    off = (w.double() * (L / G) - 1).abs().max().item()
    assert off <= 400 * 2.0 ** -24, off
    assert binding.device_error() == 0


@pytest.mark.parametrize("page", [0, 16])
@pytest.mark.parametrize("D,G,n", [(64, 4, 1), (128, 8, 1), (128, 4, 3), (256, 6, 2)])
def test_every_token_has_its_own_scale(D, G, n, page):
    """Scales of neighbouring tokens 64 times apart, over many rounds of the ring of keys: a scale of another token
    shows."""
    lens = [6000, 1, 333, 4097]
    c = Cache(D + G, lens, 6000, 2, D, page, names="k", int8=True)
    far = torch.where(torch.arange(6000, device="cuda") % 2 == 0, 2.0 ** -12, 2.0 ** -6)
    s = (torch.rand(4, 2, 6000, generator=c.gen, device="cuda") + 0.5) * far
    c.put_numbers("ks", s)
    q = randn(c.gen, 4, n, 2 * G, D)
    if page:
        got = c.numbers_back(binding.kv_weights_int8_paged(q, c.kp, c.ksp, None, c.table, c.seq_lens, c.cap))
    else:
        got = binding.kv_weights_int8_contig(q, c.k, c.ks, None, c.seq_lens)
    for b, L in enumerate(lens):
        check(got[b, :, :L], q[b], c.values("k", b), D ** -0.5, c.values("k", b))
    assert binding.device_error() == 0
