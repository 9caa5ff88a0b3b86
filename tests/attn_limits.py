"""How far the decode kernels' attention may be from float64, from their
arithmetic, per output element.

  logits     products of 16-bit values are exact in fp32; their sum of D terms
             rounds D times by 2^-23 of at most sum |q k| each (the tensor
             cores may truncate), so a scaled logit is off by at most
             delta = scale D 2^-23 max_j sum_d |q_d k_jd|, plus 2^-22 of itself
             for the scale's and the exponent's roundings;
  weights    relative error 2 delta from the logits (numerator and
             normaliser), plus the rounding of p to the product's type: fp16
             2^-11, bf16 as two parts 2^-15 (both counted twice), plus the
             exponential's 2^-21;
  sums       n + 64 additions in fp32, each 2^-23 of sum p |v| (blocks are
             summed 16 rows at a time and merged over warps and pieces);
  output     one rounding to its type, eps / 2, or half its smallest step.
"""
from __future__ import annotations

import numpy as np

EPS = {"f16": 2.0 ** -10, "bf16": 2.0 ** -7}
TINY = {"f16": 2.0 ** -25, "bf16": 2.0 ** -134}


def attend(q, k, v, scale: float, dtype: str, p16: str | None = None):
    """(attention of q [D] over k, v [n, D] in float64, limit of the error)."""
    if len(k) == 0:
        return np.zeros(q.shape), np.zeros(q.shape)
    logit = k @ q * scale
    w = np.exp(logit - logit.max())
    w /= w.sum()
    ref = w @ v
    mass = w @ np.abs(v)
    delta = abs(scale) * len(q) * 2.0 ** -23 * (np.abs(k) @ np.abs(q)).max() + 2.0 ** -22 * np.abs(logit).max()
    p_err = 2 * (2.0 ** -11 if (p16 or dtype) == "f16" else 2.0 ** -15)
    rel = 2 * delta + p_err + 2.0 ** -20 + (len(k) + 64) * 2.0 ** -23
    slack = mass * rel
    return ref, slack + (np.abs(ref) + slack) * EPS[dtype] / 2 + TINY[dtype]
