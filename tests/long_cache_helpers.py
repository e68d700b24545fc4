"""Caches for the tests of prefix attention, selected blocks, weights and eviction: the same tokens contiguous and in
shuffled pages, with NaN wherever no token lies."""
import numpy as np
import torch


def lens_of(*n):
    return torch.tensor(n, dtype=torch.int32, device="cuda")


def randn(gen, *shape, dtype=torch.bfloat16):
    return torch.randn(shape, generator=gen, device="cuda").to(dtype)


def f64(t):
    return t.double().cpu().numpy()


class Cache:
    """rows {name: [B, cap, H, D]}, contiguous; page > 0: also pools and a table, pages in random order."""

    def __init__(self, seed, lens, cap, H, D, page=0, names="kv", int8=False, spare=2):
        self.gen = torch.Generator(device="cuda").manual_seed(seed)
        self.lens, self.cap, self.page, self.H, self.D, self.int8 = list(lens), cap, page, H, D, int8
        B = len(self.lens)
        self.B, self.seq_lens = B, lens_of(*lens)
        live = [min(max(L, 0), cap) for L in lens]
        self.live = live
        if page:
            need = [-(-L // page) for L in live]
            order = np.random.default_rng(seed).permutation(sum(need) + spare)
            table, at = np.full((B, max(1, -(-cap // page))), -1, np.int32), 0
            for b, n in enumerate(need):
                table[b, :n] = order[at:at + n]
                at += n
            self.pages = sum(need) + spare
            self.table = torch.from_numpy(table).cuda()
        for x in names:
            self.put(x, torch.randint(-127, 128, (B, cap, H, D), generator=self.gen, device="cuda", dtype=torch.int8)
                     if int8 else randn(self.gen, B, cap, H, D))
            if int8:
                self.put_numbers(x + "s", torch.rand(B, H, cap, generator=self.gen, device="cuda") * 0.02 + 0.01)

    def places(self):
        """(sequence, token, page, row) of every token."""
        for b, L in enumerate(self.live):
            for j in range(-(-L // self.page)):
                yield b, j * self.page, min(L, (j + 1) * self.page), int(self.table[b, j])

    def put(self, name, rows):
        """Rows [B, cap, H, D], then the NaN and the pool."""
        rows = rows.clone()
        for b, L in enumerate(self.live):
            rows[b, L:] = 0x55 if self.int8 else float("nan")
        setattr(self, name, rows)
        if self.page:
            pool = torch.full((self.pages, self.page, self.H, self.D), 0x55 if self.int8 else float("nan"),
                              dtype=rows.dtype, device="cuda")
            for b, t0, t1, page in self.places():
                pool[page, :t1 - t0] = rows[b, t0:t1]
            setattr(self, name + "p", pool)

    def put_numbers(self, name, x):
        """Numbers [B, H, cap], fp32."""
        x = x.clone()
        for b, L in enumerate(self.live):
            x[b, :, L:] = float("nan")
        setattr(self, name, x)
        if self.page:
            pool = torch.full((self.pages, self.H, self.page), float("nan"), device="cuda")
            for b, t0, t1, page in self.places():
                pool[page, :, :t1 - t0] = x[b, :, t0:t1]
            setattr(self, name + "p", pool)

    def numbers_back(self, pool, n=None):
        """A pool of numbers as [B, H, cap], NaN where no token lies."""
        out = torch.full((self.B, self.H, self.cap), float("nan"), device="cuda")
        for b, t0, t1, page in self.places():
            out[b, :, t0:t1] = pool[page, :, :t1 - t0]
        return out

    def rows_back(self, pool):
        out = torch.zeros((self.B, self.cap, self.H, self.D), dtype=pool.dtype, device="cuda")
        for b, t0, t1, page in self.places():
            out[b, t0:t1] = pool[page, :t1 - t0]
        return out

    def values(self, name, b):
        """A sequence's rows in float64."""
        L = self.live[b]
        y = f64(getattr(self, name)[b, :L])
        return y * f64(getattr(self, name + "s")[b, :, :L]).T[..., None] if self.int8 else y


def score_error(q, k, scale, D):
    """Bound of a score's error: D / 16 MMAs in fp32 add 17 terms each, cut off at 2^-23 of |q| |k| at most, and the
    scale to log2 units and exp2 round by 2^-22 of a score."""
    top = np.sqrt((q ** 2).sum(-1).max(initial=0.0)) * np.sqrt((k ** 2).sum(-1).max(initial=0.0)) * abs(scale)
    return top * (D / 16 * 17 * 2.0 ** -23 + 2.0 ** -21) + 2.0 ** -21


def check_attention(got, want, mass, e):
    """A weight is off by its rounding to bf16 (2^-8 of it at most) and twice its score's error e; the result is
    rounded to bf16 (2^-8 of it).  The sum of the weights is taken before their rounding."""
    err = np.abs(got - want)
    tol = (2.0 ** -8 + 2 * e + 2.0 ** -16) * mass + 2.0 ** -8 * np.abs(want)
    assert np.isfinite(got).all()
    assert (err <= tol).all(), f"{err.max():.3e}, {(err - tol).max():.3e} over the bound"
