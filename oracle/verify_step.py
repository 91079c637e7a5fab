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


def sample_order(x):
    """Candidate columns of one row of logits: by falling value, then rising
    column; neither NaN nor -inf."""
    x = np.asarray(x, np.float64)
    cols = np.flatnonzero(x > -np.inf)
    return cols[np.lexsort((cols, -x[cols]))]


def sample_weights(x, order, T):
    """Weights of the ordered candidates."""
    v = np.asarray(x, np.float64)[order]
    if np.isinf(v[0]):
        return (v == v[0]).astype(np.float64)
    with np.errstate(over="ignore", invalid="ignore"):
        return np.exp((v - v[0]) / T)


def sample_row(x, u, T, top_k=0, top_p=1.0, min_p=0.0):
    """(column, logprob) of one row: the definition, on sorted columns."""
    order = sample_order(x)
    if order.size == 0:
        return 0, 0.0
    if not T > 0:
        return int(order[0]), 0.0
    w = sample_weights(x, order, T)
    n = order.size
    if top_k > 0:
        n = min(n, int(top_k))
    if top_p < 1:
        need = top_p * w[:n].sum()
        before = np.concatenate([[0.0], np.cumsum(w[:n])[:-1]])
        n_p = int(np.count_nonzero(before < need))
    else:
        n_p = n
    n = max(1, min(n, n_p, int(np.count_nonzero(w >= min(min_p, 1.0))) if min_p > 0 else n))
    cum = np.cumsum(w[:n])
    u = 0.0 if not u > 0 else min(float(u), 1 - 2.0 ** -24)
    m = min(int(np.count_nonzero(cum <= u * cum[-1])), n - 1)
    return int(order[m]), float(np.log(w[m] / cum[-1]))


def accepted_prefix(tokens, draft):
    """Per sequence the drafted tokens that equal the sampled ones in front."""
    out = []
    for t, d in zip(np.asarray(tokens), np.asarray(draft)):
        n = 0
        while n < len(d) and t[n] == d[n]:
            n += 1
        out.append(n)
    return np.array(out)


def sink_attention(q, k, v, seq_len, q_pos, window, sinks, scale):
    """Windowed attention of one sequence whose first `sinks` positions stay
    visible.

    q [q_len, Hq, D], k and v [Hkv, L, D].  Returns (out, lse, absv, mag): per
    row and head the result, and for error bounds the weighted sum of |v| per
    dim and the largest of scale * sum_d |q_d k_jd| over its visible keys.
    """
    q, k, v = (np.asarray(a, np.float64) for a in (q, k, v))
    q_len, Hq, D = q.shape
    Hkv, L = k.shape[:2]
    out, absv = np.zeros((q_len, Hq, D)), np.zeros((q_len, Hq, D))
    lse, mag = np.full((q_len, Hq), -np.inf), np.zeros((q_len, Hq))
    for i in range(q_len):
        p = q_pos + i
        js = [j for j in range(max(0, min(p + 1, seq_len, L))) if j > p - window or j < sinks]
        if not js:
            continue
        for h in range(Hq):
            kk, vv = k[h // (Hq // Hkv)][js], v[h // (Hq // Hkv)][js]
            s = scale * (kk @ q[i, h])
            m = s.max()
            e = np.exp(s - m)
            out[i, h] = e @ vv / e.sum()
            absv[i, h] = e @ np.abs(vv) / e.sum()
            lse[i, h] = m + np.log(e.sum())
            mag[i, h] = (np.abs(kk) @ np.abs(q[i, h])).max() * abs(scale)
    return out, lse, absv, mag
