"""fp64 definitions of the 8-bit KV cache and of token log probabilities.

TEST INFRASTRUCTURE ONLY, like the rest of this package; shares no code with
the CUDA library.  Plain numpy on float64 arrays.
"""
import math

import numpy as np


def _values():
    v = np.empty(256)
    for c in range(256):
        e, f = (c >> 3) & 15, c & 7
        v[c] = f * 2.0 ** -9 if e == 0 else (8 + f) * 2.0 ** (e - 10)
        if c & 127 == 127:
            v[c] = np.nan
        if c & 128:
            v[c] = -v[c]
    return v


# the 256 values of e4m3: sign, 4 exponent bits (bias 7), 3 fraction bits;
# exponent 0 counts in 2^-9, all ones is NaN
E4M3 = _values()
E_MIN, E_MAX = -50, 50


def quantise_row(x):
    """(e4m3 codes, exponent) of one row of D values."""
    x = np.asarray(x, np.float64)
    fin = np.isfinite(x)
    a = np.abs(x[fin]).max() if fin.any() else 0.0
    e = next((k for k in range(E_MIN, E_MAX + 1) if a <= 448.0 * 2.0 ** k), E_MAX)
    y = np.where(fin, x, 0.0) * 2.0 ** -e
    y = np.clip(y, -448.0, 448.0)
    steps = E4M3[:127]
    hi = np.clip(np.searchsorted(steps, np.abs(y)), 1, 126)
    up, down = steps[hi] - np.abs(y), np.abs(y) - steps[hi - 1]
    code = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, hi - 1)
    code = np.where(np.signbit(y), code | 128, code)
    return np.where(fin, code, 127).astype(np.uint8), e


def row_values(codes, e):
    return E4M3[np.asarray(codes)] * 2.0 ** np.asarray(e, np.float64)[..., None]


def attention(q, k, v, seq_len, q_pos, window, scale, dims=8):
    """One sequence: q [q_len, Hq, D], k and v [Hkv, L, D] (the values).

    Returns out [q_len, Hq, D], lse [q_len, Hq], and per row what the bounds
    on rounding errors are made of: the summed magnitude of the largest score
    (|q||k| over the dims), sum_j w_j |v_j| per dim, the keys seen."""
    q_len, Hq, D = q.shape
    Hkv, L = k.shape[:2]
    out = np.zeros((q_len, Hq, D))
    lse = np.full((q_len, Hq), -np.inf)
    mag, wv, seen = np.zeros((q_len, Hq)), np.zeros((q_len, Hq, D)), np.zeros((q_len, Hq))
    for i in range(q_len):
        p = q_pos + i
        js = np.arange(max(0, p - window + 1), min(p + 1, seq_len, L))
        if js.size == 0:
            continue
        for h in range(Hq):
            g = h // (Hq // Hkv)
            s = scale * (k[g, js] @ q[i, h])
            m = s.max()
            w = np.exp(s - m)
            lse[i, h] = m + np.log(w.sum())
            w = w / w.sum()
            out[i, h] = w @ v[g, js]
            mag[i, h] = abs(scale) * (np.abs(k[g, js]) @ np.abs(q[i, h])).max()
            wv[i, h] = w @ np.abs(v[g, js])
            seen[i, h] = js.size
    return out, lse, mag, wv, seen


def logprob_row(x, token, T=1.0, top=0, keep=None):
    """(logprob, rank, entropy, top tokens, top logprobs) of one row."""
    x = np.asarray(x, np.float64)
    x = np.where(np.isnan(x), -np.inf, x)
    if not T > 0:
        T = 1.0
    V = x.size
    order = np.lexsort((np.arange(V), -x))
    m = x.max()
    if m == -np.inf:
        lp, ent = np.full(V, -np.inf), 0.0
    else:
        y = np.where(x == m, 0.0, x - m) / T if np.isinf(m) else (x - m) / T
        lp = y - math.log(np.exp(y).sum())
        p = np.exp(lp)
        ent = -float((p[p > 0] * lp[p > 0]).sum())
    if keep is None:
        col = int(token) if 0 <= token < V else None
    else:
        at = np.flatnonzero(np.asarray(keep) == token)
        col = int(at[0]) if at.size and token >= 0 else None
    names = order[:top] if keep is None else np.asarray(keep)[order[:top]]
    if col is None:
        return -math.inf, 0, ent, names, lp[order[:top]]
    return float(lp[col]), int(np.flatnonzero(order == col)[0]) + 1, ent, names, lp[order[:top]]
