"""Rotary positions in float64: the pairs of the first ``rot`` elements of a
head turn by position times frequency, as complex numbers.

The frequencies are base^(-2 i / rot), scaled for a longer context linearly
("linear": every position divided by the factor), by a larger base ("base"),
by a ramp between frequencies that are kept and frequencies that are divided
("ramp", by pair index), or by the same choice per wavelength ("wavelength").
"""
from __future__ import annotations

import numpy as np


def frequencies(rot: int, base: float = 10000.0, scaling: str = "none", factor: float = 1.0,
                original_context: float = 8192.0, low_turns: float = 1.0, high_turns: float | None = None):
    """(radians per position [rot / 2], amplitude)."""
    i = np.arange(rot // 2)
    if scaling == "base":
        base = base * factor ** (rot / (rot - 2))
    w = np.exp(-2.0 * i / rot * np.log(base))
    if scaling in ("none", "base"):
        return w, 1.0
    if scaling == "linear":
        return w / factor, 1.0
    if scaling == "ramp":
        high = 32.0 if high_turns is None else high_turns
        # the (fractional) pair that makes n full turns in the original context
        pair = [rot / 2 * np.log(original_context / (2 * np.pi * n)) / np.log(base) for n in (high, low_turns)]
        first, last = max(np.floor(pair[0]), 0.0), min(np.ceil(pair[1]), rot - 1.0)
        divided = np.clip((i - first) / max(last - first, 0.001), 0.0, 1.0)
        return w * (1 - divided + divided / factor), 1.0 + 0.1 * np.log(factor)
    if scaling == "wavelength":
        high = 4.0 if high_turns is None else high_turns
        n = original_context / (2 * np.pi / w)
        kept = np.clip((n - low_turns) / (high - low_turns), 0.0, 1.0)
        return w * (kept + (1 - kept) / factor), 1.0
    raise ValueError(scaling)


def rotate(x, positions, freq, amplitude: float, layout: str):
    """x [T, H, D] turned at ``positions`` [T]; elements from 2 len(freq) on pass through."""
    x = np.asarray(x, dtype=np.float64)
    half = len(freq)
    angle = np.asarray(positions, dtype=np.float64)[:, None, None] * freq
    turn = amplitude * np.exp(1j * angle)
    out = x.copy()
    if layout == "half":
        z = (x[..., :half] + 1j * x[..., half:2 * half]) * turn
        out[..., :half], out[..., half:2 * half] = z.real, z.imag
    else:
        z = (x[..., 0:2 * half:2] + 1j * x[..., 1:2 * half:2]) * turn
        out[..., 0:2 * half:2], out[..., 1:2 * half:2] = z.real, z.imag
    return out
