"""Plain fp64 CPU oracle for latent attention (test infrastructure only; the CUDA library
never calls it and shares no code with it).

One cached row c_t = [latent (R), rotated part (P)] a token is shared by all heads.

absorbed:  s_t = scale <q, c_t>, out = sum_t softmax(s)_t c_t[:R]; query token i of the last
           q_len sees the first L - q_len + 1 + i tokens; one that sees none gives zeros.
expanded:  head h's key is [k_nope[t, h], k_rope[t]] and its value v[t, h], with k_nope and v
           linear in the latent; the same causal attention.
"""
from __future__ import annotations

import numpy as np

__all__ = ["absorbed", "expanded", "gather_rows"]


def gather_rows(pool, table_row, L, page_size):
    """The first L rows of a sequence from its pages."""
    t = np.arange(L)
    return pool[table_row[t // page_size], t % page_size]


def _attend(scores, values, L, q_len):
    """scores [q_len, ..., L], values [L, D] or with matching leading axes -> ([q_len, ..., D], weights)."""
    seen = L - q_len + 1 + np.arange(q_len)
    hide = np.arange(L) >= seen[:, None]
    hide = hide.reshape((q_len,) + (1,) * (scores.ndim - 2) + (L,))
    s = np.where(hide, -np.inf, scores)
    top = s.max(axis=-1, keepdims=True) if L else np.zeros(s.shape[:-1] + (1,))
    w = np.where(hide, 0.0, np.exp(s - np.where(np.isfinite(top), top, 0.0)))
    den = w.sum(axis=-1, keepdims=True)
    return np.where(den > 0, w / np.where(den > 0, den, 1.0), 0.0)


def absorbed(q, rows, R, scale, spread=False):
    """q [q_len, H, W], rows [L, W] (float64) -> [q_len, H, R]; with spread also sum_t p_t |c_t| (same shape)."""
    L = rows.shape[0]
    p = _attend(scale * np.einsum("ihw,tw->iht", q, rows), rows, L, q.shape[0])
    out = np.einsum("iht,tr->ihr", p, rows[:, :R])
    return (out, np.einsum("iht,tr->ihr", p, np.abs(rows[:, :R]))) if spread else out


def expanded(q, k_nope, k_rope, v, scale, spread=False):
    """q [q_len, H, D + P], k_nope/v [L, H, D], k_rope [L, P] (float64) -> [q_len, H, D]."""
    L, H, D = k_nope.shape
    s = np.einsum("ihd,thd->iht", q[..., :D], k_nope) + np.einsum("ihd,td->iht", q[..., D:], k_rope)
    p = _attend(scale * s, v, L, q.shape[0])
    out = np.einsum("iht,thd->ihd", p, v)
    return (out, np.einsum("iht,thd->ihd", p, np.abs(v))) if spread else out
