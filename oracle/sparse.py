"""Block-sparse decode in float64: bounds of a block's keys, scores of the
blocks, the choice of blocks, and attention over the chosen ones."""
from __future__ import annotations

import numpy as np


def block_bounds(keys: np.ndarray, rows: int):
    """(minimum, maximum) over the first ``rows`` rows of keys [16, D]."""
    return keys[:rows].min(axis=0), keys[:rows].max(axis=0)


def block_score(q_group: np.ndarray, lo: np.ndarray, hi: np.ndarray, scale: float) -> float:
    """The largest scaled logit that a key between lo and hi could have with
    any query head of q_group [G, D]."""
    return scale * float(np.maximum(q_group * lo, q_group * hi).sum(axis=1).max())


def select_blocks(scores, n_blocks: int, first: int, last: int, budget: int) -> list[int]:
    """Ascending list of at most ``budget`` of the blocks 0..n_blocks-1."""
    if n_blocks <= budget:
        return list(range(n_blocks))
    chosen = set(range(first)) | set(range(n_blocks - last, n_blocks))

    def rank(i):
        s = float(scores[i])
        return (0, 0.0, i) if np.isnan(s) else (1, -s, i)     # NaN above every number
    rest = sorted((i for i in range(n_blocks) if i not in chosen), key=rank)
    return sorted(chosen | set(rest[:budget - len(chosen)]))


def token_positions(listed, n_tokens: int) -> np.ndarray:
    """Positions of the tokens in the listed blocks (negative entries are
    skipped; a block listed twice counts twice)."""
    pos = [np.arange(16 * int(i), min(16 * int(i) + 16, n_tokens)) for i in listed if int(i) >= 0]
    return np.concatenate(pos) if pos else np.zeros(0, dtype=np.int64)
