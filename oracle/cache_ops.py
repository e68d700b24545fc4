"""Plain CPU oracle for rotary positions, cache writes and cache reads (test
infrastructure only; the CUDA library never calls it and shares no code with it).

Rotary positions: pair j of a head, elements (a, b), is the complex number a + ib times
magnitude exp(i p w_j), or the conjugate of that for the gradient, in float64.

Cache writes: new token i of sequence b is position L_b - q_len + i; positions below 0 or
at or past the capacity are not written.  int8 rows: scale = max|x| / 127 in float32 (1 for
a row of zeros), values rint(x / scale); a row with a non-finite element gets a NaN scale
and zeros.  Reads widen int8 * scale in float32 and round once to bf16.
"""
from __future__ import annotations

import numpy as np

from .decode_attention import round_to_bf16

__all__ = ["rotate", "quantize", "new_positions", "write", "read"]


def rotate(x, positions, inv_freq, offset=0, interleaved=False, magnitude=1.0, backward=False):
    """x [..., H, D] float64, positions [...] -> the rotated heads, float64."""
    x = np.array(x, dtype=np.float64)
    np_ = len(inv_freq)
    j = np.arange(np_)
    a, b = (offset + 2 * j, offset + 2 * j + 1) if interleaved else (offset + j, offset + np_ + j)
    angle = np.asarray(positions, dtype=np.float64)[..., None] * np.asarray(inv_freq, dtype=np.float64)
    turn = magnitude * np.exp(1j * (-angle if backward else angle))[..., None, :]
    z = (x[..., a] + 1j * x[..., b]) * turn
    x[..., a], x[..., b] = z.real, z.imag
    return x


def quantize(x):
    """Rows (last axis) of float32 or float64 -> (int8, float32 scale)."""
    x32 = np.asarray(x).astype(np.float32)
    top = np.abs(x32).max(axis=-1)
    bad = ~np.isfinite(x32).all(axis=-1)
    with np.errstate(all="ignore"):
        scale = np.where(top > 0, np.maximum(top / np.float32(127), np.finfo(np.float32).tiny), np.float32(1))
        q = np.clip(np.rint(x32 / scale[..., None].astype(np.float32)), -127, 127)
    q = np.where(bad[..., None], 0, q).astype(np.int8)
    return q, np.where(bad, np.nan, scale).astype(np.float32)


def new_positions(seq_lens, q_len):
    """[B, q_len] positions of the new tokens."""
    return np.asarray(seq_lens, np.int64)[:, None] - q_len + np.arange(q_len)


def write(cache, rows, seq_lens, cap, table=None, page_size=0):
    """cache[...] = rows [B, q_len, ...] at the new tokens' places.  A contiguous cache is
    [B, max_ctx, ...]; pages are [num_pages, page_size, ...].  Returns (a new array, whether a
    token lay past the capacity, whether a page was outside the pool)."""
    out = cache.copy()
    late = bad = False
    for b, line in enumerate(new_positions(seq_lens, rows.shape[1])):
        for i, p in enumerate(line):
            if p < 0:
                continue
            if p >= cap:
                late = True
            elif table is None:
                out[b, p] = rows[b, i]
            else:
                page = int(table[b, p // page_size])
                if 0 <= page < cache.shape[0]:
                    out[page, p % page_size] = rows[b, i]
                else:
                    bad = True
    return out, late, bad


def read(out, values, seq_lens, cap, n, starts=None, table=None, page_size=0, scales=None):
    """bf16 bits [B, n, H, D]: `out` with the cache's tokens in place.  values: bf16 bits or int8 (scales:
    [B or pages, H, tokens])."""
    out = out.copy()
    B = len(seq_lens)
    for b in range(B):
        L = min(int(seq_lens[b]), cap)
        for i in range(n):
            p = (0 if starts is None else int(starts[b])) + i
            if p < 0 or p >= L:
                continue
            slab, at = (b, p) if table is None else (int(table[b, p // page_size]), p % page_size)
            if not 0 <= slab < values.shape[0]:
                continue
            v = values[slab, at]
            if scales is not None:
                v = round_to_bf16((v.astype(np.float32) * scales[slab, :, at][:, None]).astype(np.float64))
            out[b, i] = v
    return out


