"""CPU oracle for rotary positions.

TEST INFRASTRUCTURE, like the rest of ``oracle/``.  numpy in float64, complex
products; it shares nothing with the CUDA path.

A pair (a, b) of a head's elements is the complex number a + i b, and a token
at position p multiplies it by rot_scale * exp(i p w) for the pair's angular
frequency w (Su et al., RoFormer, arXiv 2104.09864).  The pairs of the rotated
part are (j, j + rot/2) or, interleaved, (2 j, 2 j + 1).  The gradient of the
map is the conjugate factor.
"""
from __future__ import annotations

import numpy as np


def frequencies(rot: int, base: float = 10000.0, scaling: str = "none", factor: float = 1.0,
                orig_len: float = 0.0, beta_fast: float = 32.0, beta_slow: float = 1.0):
    """Angular frequencies [rot / 2] (radians per position) and rot_scale."""
    j = np.arange(rot // 2, dtype=np.float64)
    if scaling == "ntk":
        base = base * factor ** (rot / (rot - 2.0))
    w = base ** (-2.0 * j / rot)
    if scaling == "linear":
        w = w / factor
    if scaling == "yarn":
        # pairs that turn often enough over the trained length keep their
        # frequency, slow ones are stretched (Peng et al., arXiv 2309.00071)
        turns = orig_len / (2.0 * np.pi / w)
        keep = np.interp(turns, [beta_slow, beta_fast], [0.0, 1.0])
        return keep * w + (1.0 - keep) * w / factor, 0.1 * np.log(factor) + 1.0
    return w, 1.0


def turns_to_frequencies(freqs) -> np.ndarray:
    """Radians per position from the table's 2^-64 turns."""
    return np.asarray(freqs).astype(np.int64).view(np.uint64).astype(np.float64) * (
        2.0 * np.pi / 2.0 ** 64)


def rope(x, positions, w, rot_scale: float = 1.0, offset: int = 0, interleaved: bool = False,
         inverse: bool = False, out_scale: float = 1.0) -> np.ndarray:
    """x [L][H][d] float64 -> the rotated array, float64."""
    x = np.asarray(x, np.float64)
    half = len(w)
    y = x.copy()
    th = np.asarray(positions, np.float64)[:, None] * np.asarray(w, np.float64)
    z = rot_scale * np.exp((-1j if inverse else 1j) * th)[:, None, :]
    if interleaved:
        a, b = offset + 2 * np.arange(half), offset + 2 * np.arange(half) + 1
    else:
        a, b = offset + np.arange(half), offset + half + np.arange(half)
    v = (x[..., a] + 1j * x[..., b]) * z
    y[..., a], y[..., b] = v.real, v.imag
    return y * out_scale
