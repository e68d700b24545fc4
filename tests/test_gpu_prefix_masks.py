"""Values of a shared prefix that are not finite reach the rows that see them and no others, whatever the number of rows
and the prefix's length."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from long_cache_helpers import Cache, f64, lens_of, randn, score_error  # noqa: E402
from oracle import long_cache as ol  # noqa: E402
from gqa_split_kv_gb300 import binding  # noqa: E402


class Behind:
    """Sequences of these lengths behind a prefix of P tokens, some of which end inside it; finite everywhere."""

    def __init__(self, seed, P, lens, n, Hq, Hkv, D, page):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.P, self.lens, self.n, self.page = P, lens, n, page
        self.q = randn(gen, len(lens), n, Hq, D)
        self.kp, self.vp = randn(gen, P, Hkv, D), randn(gen, P, Hkv, D)
        rest = max(max(lens) - P, 0) + 5
        self.k, self.v = (randn(gen, len(lens), rest, Hkv, D) for _ in "kv")
        self.seq_lens = lens_of(*lens)
        if page:
            self.c = Cache(seed, [P + rest] * len(lens), P + rest, Hkv, D, page)
            self.prefix_table = self.c.table[0, :-(-P // page)].contiguous()

    def run(self):
        if not self.page:
            return binding.prefix_attn_contig(self.q, self.kp, self.vp, self.k, self.v, self.seq_lens)
        pools = []
        for head, own, name in ((self.kp, self.k, "k"), (self.vp, self.v, "v")):
            rows = torch.cat((head[None].expand(len(self.lens), -1, -1, -1), own), 1)
            self.c.put(name, rows)
            pools.append(getattr(self.c, name + "p"))
        return binding.prefix_attn_paged(self.q, *pools, self.prefix_table, self.P, self.c.table, self.seq_lens,
                                         self.c.cap)

    def seen(self):
        """[B, n] tokens that each query token sees."""
        return np.array([[max(L - self.n + 1 + i, 0) for i in range(self.n)] for L in self.lens])


    def exact(self):
        """The finite prefix's and rests' results and their tolerances: a weight is off by its rounding to bf16 (2^-8 of it)
        and twice its score's error, the result by its rounding."""
        scale, want, tol = self.q.shape[-1] ** -0.5, [], []
        for b, L in enumerate(self.lens):
            k, v = (np.concatenate((f64(x), f64(y[b])))[:L] for x, y in ((self.kp, self.k), (self.vp, self.v)))
            q = f64(self.q[b])
            out, mass = ol.attend(q, k, v, scale)
            want.append(out)
            tol.append((2.0 ** -8 + 2 * score_error(q, k, scale, q.shape[-1]) + 2.0 ** -16) * mass + 2.0 ** -8 * np.abs(out))
        return np.array(want), np.array(tol)


def ends(rng, P, B, n):
    """Lengths inside the prefix, at its end, past it, and none."""
    lens = [int(x) for x in rng.integers(1, P + 40, B)]
    lens[0], lens[1], lens[2], lens[3], lens[-1] = P + 30, 0, P, P // 3 + n, P + n
    return lens


@pytest.mark.parametrize("page", [0, 16, 48])
@pytest.mark.parametrize("P,B,n,Hq,Hkv,D", [(300, 5, 1, 8, 2, 128), (3000, 5, 1, 32, 2, 128), (700, 40, 1, 16, 2, 64),
                                            (1000, 24, 2, 12, 2, 256), (130, 70, 4, 8, 1, 128), (2500, 9, 3, 24, 4, 256),
                                            (64, 30, 5, 4, 1, 64)])
def test_values_reach_the_rows_that_see_them(P, B, n, Hq, Hkv, D, page):
    rng = np.random.default_rng(P + B)
    lens = ends(rng, P, B, n)
    s = Behind(P + D, P, lens, n, Hq, Hkv, D, page)
    (want, tol), seen = s.exact(), s.seen()
    assert (np.abs(f64(s.run()) - want) <= tol).all()
    inside = sorted({int(x) for x in seen.ravel() if 0 < x < P})
    G = Hq // Hkv
    for t in {P - 1, P // 2, inside[0] - 1, inside[len(inside) // 2], 0}:
        for bad in (float("inf"), float("nan")):
            keep, next_t = s.vp.clone(), min(t + 1, P - 1)
            s.vp[t, Hkv - 1, 3:9] = bad
            s.vp[next_t, Hkv - 1, D - 1] = -float("inf")
            got = f64(s.run())
            touched = np.zeros(got.shape, bool)
            touched[:, :, -G:, 3:9] = (seen > t)[..., None, None]
            touched[:, :, -G:, D - 1] = (seen > next_t)[..., None]
            assert (np.isfinite(got) == ~touched).all(), (t, bad, np.argwhere(np.isfinite(got) == touched)[:4])
            assert (np.abs(got - want) <= tol)[~touched].all(), (t, bad)
            s.vp.copy_(keep)
    assert binding.device_error() == 0


@pytest.mark.parametrize("P,B,n,Hq,Hkv,D", [(700, 40, 1, 16, 2, 64), (3000, 5, 1, 32, 2, 128), (1000, 24, 2, 12, 2, 256)])
def test_signs_and_keys(P, B, n, Hq, Hkv, D):
    """An infinity keeps its sign, two of different signs are NaN, and keys of NaN reach no row before them."""
    lens = ends(np.random.default_rng(B), P, B, n)
    s = Behind(B, P, lens, n, Hq, Hkv, D, 0)
    s.q.zero_()  # equal weights of 1, exact in bf16: a result is off by its own rounding, 2^-8 of it at most, on each side
    clean, seen = s.run(), s.seen()
    t = sorted({int(x) for x in seen.ravel() if 0 < x < P})[0]
    s.vp[t, :, 0], s.vp[t, :, 1], s.vp[t, :, 2] = float("inf"), -float("inf"), float("inf")
    s.vp[min(t + 1, P - 1), :, 2] = -float("inf")
    out = s.run()
    sees, both = (torch.from_numpy(seen > x).cuda()[..., None] for x in (t, min(t + 1, P - 1)))
    assert torch.equal(torch.isposinf(out[..., 0]), sees.expand(-1, -1, Hq))
    assert torch.equal(torch.isneginf(out[..., 1]), sees.expand(-1, -1, Hq))
    assert torch.equal(torch.isnan(out[..., 2]), both.expand(-1, -1, Hq))
    assert (out[..., 3:].float() - clean[..., 3:].float()).abs().max() <= 2.0 ** -7 * clean.float().abs().max()
    s = Behind(B, P, lens, n, Hq, Hkv, D, 0)
    clean = s.run()
    s.kp[t] = float("nan")
    out = s.run()
    rows = torch.from_numpy(seen <= t).cuda()
    assert torch.equal(out[rows], clean[rows]) and torch.isnan(out[~rows]).all()
    assert binding.device_error() == 0
