"""The windowed attention over an 8-bit cache in 64 bits, with what bounds on its
rounding errors are made of (shared by the tests of that attention)."""
import numpy as np

import oracle.kv8 as kv8


def attention(q, k8, v8, ke, ve, seq_len, q_pos, window, scale):
    """One sequence: q [q_len, Hq, D] values, k8 and v8 [Hkv, L, D] e4m3 codes, ke and
    ve [Hkv, L] exponents.

    Returns out [q_len, Hq, D], lse [q_len, Hq] and per row
      mag   the largest scale * sum |q||k| of a visible key; (D + 16) 2^-24 of it bounds
            a score's error, so that of q elements below 2^-14 of their row's largest
            (2^-21 of that largest, times |k|) is added as that many times as much
      wv    sum_j w_j |v_j| per dim
      top   the largest w_j * 448 * 2^e_j
      seen  the keys it sees."""
    q_len, Hq, D = q.shape
    Hkv, L = k8.shape[:2]
    out, wv = np.zeros((q_len, Hq, D)), np.zeros((q_len, Hq, D))
    lse = np.full((q_len, Hq), -np.inf)
    mag, top, seen = (np.zeros((q_len, Hq)) for _ in range(3))
    first, end = max(0, q_pos - window + 1), min(seq_len, L, q_pos + q_len)
    if end <= first:
        return out, lse, mag, wv, top, seen
    for g in range(Hkv):
        k = kv8.row_values(k8[g, first:end], ke[g, first:end])
        v = kv8.row_values(v8[g, first:end], ve[g, first:end])
        row = 448.0 * 2.0 ** ve[g, first:end].astype(np.float64)
        for i in range(q_len):
            p = q_pos + i
            see = slice(max(p - window + 1 - first, 0), max(min(p + 1, end) - first, 0))
            if see.stop <= see.start:
                continue
            for h in range(g * (Hq // Hkv), (g + 1) * (Hq // Hkv)):
                s = scale * (k[see] @ q[i, h])
                m = s.max()
                w = np.exp(s - m)
                lse[i, h] = m + np.log(w.sum())
                w /= w.sum()
                out[i, h], wv[i, h] = w @ v[see], w @ np.abs(v[see])
                big = np.abs(q[i, h]).max()
                off = np.where(np.abs(q[i, h]) < 2.0 ** -14 * big, 2.0 ** -21 * big, 0.0)
                mag[i, h] = abs(scale) * (np.abs(k[see]) @ (np.abs(q[i, h]) +
                                                            off * 2.0 ** 24 / (D + 16))).max()
                top[i, h], seen[i, h] = (w * row[see]).max(), see.stop - see.start
    return out, lse, mag, wv, top, seen
