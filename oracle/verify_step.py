"""fp64 definitions of the operators around the windowed attention.

TEST INFRASTRUCTURE ONLY, like the rest of this package; shares no code with
the CUDA library.  Plain numpy on float64 arrays, one loop per definition.
"""
import numpy as np


def norm_rope(x, weight, eps, inv_freq, pos, interleaved=False):
    """RMS norm and rotation of head rows.

    x [tokens, heads, D], weight [D] or None (no norm), inv_freq [rot / 2] or
    None, pos [tokens].  Returns (y, size): the result and, per element, the
    magnitude |a| + |b| its rounding errors scale with.
    """
    x = np.asarray(x, dtype=np.float64)
    y = x.copy()
    if weight is not None:
        y = x / np.sqrt((x * x).mean(axis=-1, keepdims=True) + eps) * np.asarray(weight, np.float64)
    size = np.abs(y)
    if inv_freq is None:
        return y, size
    half = len(inv_freq)
    # (an angle of 2^31 positions keeps 53 - 31 bits below a radian: the tests
    # of far positions allow for it)
    ang = np.asarray(pos, np.float64)[:, None, None] * np.asarray(inv_freq, np.float64)
    c, s = np.cos(ang), np.sin(ang)
    out = y.copy()
    ia, ib = ((slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved else
              (slice(0, half), slice(half, 2 * half)))
    a, b = y[..., ia], y[..., ib]
    out[..., ia], out[..., ib] = a * c - b * s, b * c + a * s
    size[..., ia] = size[..., ib] = np.abs(a) + np.abs(b)
    return out, size
