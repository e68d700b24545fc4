"""Plain fp64 CPU oracle for attention over long caches (test infrastructure only; the CUDA library never calls it
and shares no code with it).

All functions take one sequence: q [n, Hq, D], keys and values [L, Hkv, D] in float64; query head h reads KV head
h / G, and query token i (the last n of L tokens) sees tokens 0 .. L - n + i.
"""
from __future__ import annotations

import numpy as np

__all__ = ["attend", "block_means", "block_scores", "select", "block_tokens", "weights", "evict"]


def _softmax(z):
    e = np.exp(z - z.max(-1, keepdims=True))
    return e / e.sum(-1, keepdims=True)


def attend(q, k, v, scale, tokens=None):
    """out [n, Hq, D] and sum_t w_t |v_t|; tokens[i][h]: the tokens that query i of KV head h may see (all if None),
    a token as often as it is named.  Rows that see nothing are zeros."""
    n, Hq, D = q.shape
    L, H = k.shape[:2]
    G = Hq // H
    out, mass = np.zeros((n, Hq, D)), np.zeros((n, Hq, D))
    for i in range(n):
        seen = L - n + 1 + i
        for h in range(H):
            t = np.arange(max(seen, 0)) if tokens is None else np.array([x for x in tokens[i][h] if x < seen], int)
            if len(t) == 0:
                continue
            w = _softmax(q[i, h * G:(h + 1) * G] @ k[t, h].T * scale)
            out[i, h * G:(h + 1) * G] = w @ v[t, h]
            mass[i, h * G:(h + 1) * G] = w @ np.abs(v[t, h])
    return out, mass


def block_means(k, block, n):
    """{j: mean key [H, D]} of the blocks that hold the last n tokens."""
    L = len(k)
    return {j: k[j * block:(j + 1) * block].mean(0) for j in range(max(L - n, 0) // block, -(-L // block))
            if L > 0 and n > 0}


def block_scores(q_i, means):
    """[H, blocks] for one query token q_i [Hq, D], means [H, blocks, D]; NaN counts as lowest."""
    H = means.shape[0]
    with np.errstate(invalid="ignore"):
        s = np.einsum("hgd,hjd->hgj", q_i.reshape(H, -1, q_i.shape[-1]), means)
    return np.where(np.isnan(s), -np.inf, s).max(1)


def select(q, means, L, block, pick, first, recent):
    """[n, H, pick] int32, ascending, -1 behind the last."""
    n, H = len(q), means.shape[0]
    out = np.full((n, H, pick), -1, np.int32)
    for i in range(n):
        pos = L - n + i
        if pos < 0:
            continue
        visible = pos // block + 1
        score = block_scores(q[i], means[:, :visible])
        for h in range(H):
            must = [j for j in range(visible) if j < first or j >= visible - recent]
            if visible > pick:
                rest = [j for j in np.argsort(-score[h], kind="stable").tolist() if j not in set(must)]
                mine = sorted(must + rest[:pick - len(must)])
            else:
                mine = list(range(visible))
            out[i, h, :len(mine)] = mine
    return out


def block_tokens(blocks_row, block):
    """Tokens of the listed blocks, a block as often as it is listed."""
    return [t for j in map(int, blocks_row) if j >= 0 for t in range(j * block, (j + 1) * block)]


def weights(q, k, scale):
    """[H, L]: the weight that each token gets, summed over the new tokens and a group's heads."""
    n, Hq, D = q.shape
    L, H = k.shape[:2]
    G = Hq // H
    out = np.zeros((H, L))
    for i in range(n):
        seen = L - n + 1 + i
        if seen <= 0:
            continue
        for h in range(H):
            out[h, :seen] += _softmax(q[i, h * G:(h + 1) * G] @ k[:seen, h].T * scale).sum(0)
    return out


def evict(w, keep, first, recent):
    """Kept positions of one sequence and head, ascending; w [L], NaN lowest."""
    L = len(w)
    if L <= keep:
        return np.arange(L)
    lo, hi = first, L - recent
    mid = np.where(np.isnan(w[lo:hi]), -np.inf, w[lo:hi])
    nan = np.isnan(w[lo:hi])
    order = np.lexsort((np.arange(hi - lo), nan, -mid))  # by weight, NaN behind -inf, then by position
    return np.sort(np.concatenate((np.arange(lo), order[:keep - first - recent] + lo, np.arange(hi, L))))
