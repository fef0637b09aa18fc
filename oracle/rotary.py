"""fp64 oracle of the rotary positions (numpy; test infrastructure only)."""
import math

import numpy as np

from oracle.softmax_attention import host64


def frequencies(rot, base=10000.0, scaling=0, factor=1.0, original=0, beta_fast=32.0,
                beta_slow=1.0):
    """Angle per position of each pair: plain (0), linear (1), changed base (2), by parts (3)."""
    i = np.arange(rot // 2, dtype=np.float64)
    if scaling == 2 and rot > 2:
        base = base * factor ** (rot / (rot - 2))
    f = base ** (-2 * i / rot)
    if scaling == 1:
        f = f / factor
    if scaling == 3:
        turns = original * f / (2 * math.pi)
        keep = np.clip((turns - beta_slow) / (beta_fast - beta_slow), 0, 1)
        f = keep * f + (1 - keep) * f / factor
    return f


def phase_words(f):
    """Frequencies as the signed 64-bit fractions of a turn that the library takes."""
    words = [int(round((x / (2 * math.pi)) % 1.0 * 2.0 ** 64)) % (1 << 64) for x in f]
    return np.array([w - (1 << 64) if w >> 63 else w for w in words], dtype=np.int64)


def rotate(x, f, positions, rot, interleaved=False, amplitude=1.0, inverse=False):
    """x [b][h][n][d] turned, positions [b][n]."""
    x = host64(x)
    y = x.copy()
    t = np.asarray(positions, dtype=np.float64)[:, None, :, None] * np.asarray(f)
    c, s = amplitude * np.cos(t), amplitude * np.sin(t) * (-1 if inverse else 1)
    p = np.arange(rot // 2)
    a, z = (2 * p, 2 * p + 1) if interleaved else (p, p + rot // 2)
    y[..., a] = x[..., a] * c - x[..., z] * s
    y[..., z] = x[..., z] * c + x[..., a] * s
    return y
