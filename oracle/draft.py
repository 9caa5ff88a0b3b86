"""Drafted tokens and bounded contexts in float64: what the tokens of a tree
see, where they sit, attention under an explicit visibility, the move of the
accepted rows, and the window rule."""
from __future__ import annotations

import numpy as np


def ancestors(parents) -> np.ndarray:
    """bool [n, n]: entry (i, j) is set where j is i or an ancestor of i
    (parents[i] < i, -1: none)."""
    n = len(parents)
    seen = np.zeros((n, n), dtype=bool)
    for i in range(n):
        j = i
        while j >= 0:
            seen[i, j] = True
            j = int(parents[j])
    return seen


def mask_words(seen: np.ndarray, words: int) -> np.ndarray:
    """Rows of bool [n, m] as int64 [n, words]: bit j % 64 of word j // 64."""
    out = np.zeros((seen.shape[0], words), dtype=np.uint64)
    for i, j in zip(*np.nonzero(seen)):
        out[i, j // 64] |= np.uint64(1) << np.uint64(j % 64)
    return out.view(np.int64)


def masked_attend(q, keys, values, seen, scale: float) -> np.ndarray:
    """softmax(scale q K^T) V over the keys that ``seen`` [m, n] allows each row
    of q [m, d]; 0 for a row that sees none.  What is not seen takes no part,
    whatever it holds."""
    out = np.zeros((q.shape[0], values.shape[1]))
    for i in range(q.shape[0]):
        at = np.flatnonzero(seen[i])
        if len(at) == 0:
            continue
        s = scale * (keys[at] @ q[i])
        p = np.exp(s - s.max())
        out[i] = (p / p.sum()) @ values[at]
    return out


def window_seen(positions, n_keys: int, window: int, sinks: int) -> np.ndarray:
    """bool [m, n_keys]: token at position p sees j <= p with j < sinks or
    p - j < window."""
    p, j = np.asarray(positions)[:, None], np.arange(n_keys)[None]
    return (j <= p) & ((j < sinks) | (p - j < window))


def tree_seen(base: int, seen: np.ndarray) -> np.ndarray:
    """Visibility over a context of base tokens and the drafted ones behind it."""
    return np.concatenate([np.ones((seen.shape[0], base), dtype=bool), seen], axis=1)


def commit(rows: np.ndarray, base: int, accepted) -> np.ndarray:
    """rows [n, ...] by position, with the accepted ones' copies from base on."""
    out = rows.copy()
    for k, a in enumerate(accepted):
        out[base + k] = rows[base + a]
    return out
