"""Sampled verification at every launch shape (clusters of 1, 2, 4 and 8 CTAs
per row, with and without the first chunk held in registers) and at the edges
of its settings, against the fp64 definition; tolerances as in
tests/test_sample_gpu.py."""
import numpy as np
import pytest
import torch

import oracle.verify_step as vs
from tests.test_sample_gpu import _check, _logits, _row_settings, _settings

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sliding_window_speculative_gb300 import build
    build.build()
    yield


def _shape(rows, V):
    """(CTAs per row, first chunk held) as the launch chooses them."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    c = 1
    while c < 8 and rows * c * 2 <= 2 * sms and (V + 14) // 8 > 1024 * c:
        c *= 2
    return c, c == 8 and rows * c <= sms


# (B, q_len, V) -> CTAs per row; the last three settle each cluster's smallest rows
TWO = [(100, 1, 100003), (38, 4, 50257), (3, 3, 12001), (1, 1, 8201), (5, 3, 16371)]
OTHERS = [(160, 1, 20011), (300, 1, 8187), (19, 4, 40009), (2, 2, 16391), (5, 3, 32753),
          (12, 3, 65537), (1, 1, 32777), (2, 4, 131071)]


def test_every_launch_shape_is_among_the_cases():
    assert {_shape(B * q, V) for B, q, V in TWO} == {(2, False)}
    assert {_shape(B * q, V) for B, q, V in TWO + OTHERS} == {
        (1, False), (2, False), (4, False), (8, False), (8, True)}


@pytest.mark.parametrize("mode", ["none", "k", "p", "m", "all"])
@pytest.mark.parametrize("B,q_len,V", TWO + OTHERS)
def test_shapes_and_filters(B, q_len, V, mode):
    x = _logits("normal", (B, q_len, V), seed=V + len(mode))
    x[::2] = _logits("peaked", x[::2].shape, seed=V)
    u = np.random.default_rng(V + 2).random((B, q_len)).astype(np.float32)
    _check(x, _settings(B, V + 1, mode), u, what=f"{B} x {q_len} x {V} {mode}")


@pytest.mark.parametrize("kind", ["ties", "special", "negative", "small", "large"])
def test_kinds_by_two_ctas(kind):
    B, V = 84, 9001
    assert _shape(B, V) == (2, False)
    x = _logits(kind, (B, 1, V), seed=5)
    u = np.random.default_rng(6).random((B, 1)).astype(np.float32)
    for mode in ("none", "all"):
        _check(x, _settings(B, 7, mode), u, what=f"{kind} {mode}")


def _check_vanishing(x, s, u, what):
    """Rows whose values all lie within 2^-22 T of 0.  The header lets each
    weigh like 0, a relative error of 2^-22 in w.  With weights in
    [w (1 - e), w (1 + e)], e = 2^-22, any sum of them is off by as much: w >= m
    decides as for some m' in m (1 +- e), a prefix reaches p of the total as
    for some p' in p (1 +- 2 e), the running weight passes u of it as for
    some u' in u (1 +- 2 e), each to first order; w / S is off by 2 e.  So every
    token between those of the borders of these ranges is right, and every
    logprob within 2 e and the usual tolerance of one of theirs."""
    import sliding_window_speculative_gb300 as swa
    e = 2.0 ** -22 * 1.01           # (the second-order terms are below 2^-43)
    dev = {k: None if v is None else torch.from_numpy(v).cuda() for k, v in s.items()}
    t, _, lp = swa.swa_sample_accept(x.cuda(), torch.from_numpy(u).cuda(), **dev)
    torch.cuda.synchronize()
    for b in range(x.shape[0]):
        row, kw = x[b, 0].double().numpy(), _row_settings(s, b)
        assert np.abs(row).max() <= 2.0 ** -22 * kw["T"] or not kw["T"] > 0
        place = np.empty(row.size, np.int64)
        place[vs.sample_order(row)] = np.arange(row.size)
        ways = []                   # the fewest and the most kept, with the least and the largest u
        for sign in (-1, 1):
            k2 = dict(kw)
            if "min_p" in kw and (sign > 0 or kw["min_p"] < 1):   # (1 and above count as 1)
                k2["min_p"] = min(kw["min_p"], 1.0) * (1 - sign * e)
            if kw.get("top_p", 1.0) < 1:
                k2["top_p"] = kw["top_p"] * (1 + 2 * sign * e)
            ways.append([vs.sample_row(row, float(u[b, 0]) * (1 + 2 * us * e), **k2)
                         for us in (-1, 1)])
        got, g = int(t[b, 0]), float(lp[b, 0])
        assert any(place[lo[0]] <= place[got] <= place[hi[0]] and
                   abs(g - lo[1]) <= 2 * e + 2.0 ** -20 * abs(lo[1]) + 2.0 ** -34
                   for lo, hi in ways), (what, b, got, g, ways)


@pytest.mark.parametrize("mode", ["none", "k", "p", "m", "all"])
def test_rows_that_outgrow_their_first_chunk_by_two_ctas(mode):
    """Each CTA has 70,001 columns and a first chunk of 32,768: what matters
    lies behind it in the first one, in the second one, or in both."""
    V, n = 140003, 84
    assert _shape(n, V) == (2, False)
    base = _logits("normal", (1, 1, V), seed=22)[0, 0]
    rows = []
    for kind in range(12):
        x = base.clone()
        if kind == 0:
            x[60000:60005] = 3.0e4
        elif kind == 1:
            x[139000:139005] = 3.0e4
        elif kind == 2:
            x[:120000] = float("-inf")
        elif kind == 3:
            x[:135000] = float("nan")
            x[140002] = float("inf")
        elif kind == 4:
            x[:] = 1.5
        elif kind == 5:
            x[:60000] = -300.0
            x[70002:130000] = -300.0
        elif kind == 6:
            x[50000:] = 7.0
        elif kind == 7:
            x[:] = float("-inf")
            x[V - 1] = -5.0
        elif kind == 8:
            x[:69000] = torch.finfo(torch.bfloat16).min
        elif kind == 9:
            x[:110000] = -1.0e6
            x[110000:] *= 1e-3
        elif kind == 10:
            x[:] = -1.0e-12
            x[69999] = 0.0
        else:
            x[:] = -1.0e30
            x[65000] = -9.0e29
        rows.append(x)
    xs = torch.stack(rows).repeat(7, 1).view(n, 1, V)
    s = _settings(n, 18, mode)
    u = np.random.default_rng(3).random((n, 1)).astype(np.float32)
    tiny = np.arange(n) % 12 == 10

    def part(rows, check):
        check(xs[torch.from_numpy(rows)], {k: None if v is None else v[rows] for k, v in s.items()},
              u[rows], what=mode)

    # (each part as many rows as all, so that two CTAs share one)
    part(np.resize(np.flatnonzero(tiny), n), _check_vanishing)
    part(np.resize(np.flatnonzero(~tiny), n), _check)


def test_lists_of_every_length_by_two_ctas():
    """From one to thousands of columns on min-p's line and above the top-k
    bound: both CTAs' parts moved together, sorted in each way, or given up."""
    n, V = 100, 120011
    assert _shape(n, V) == (2, False)
    x = _logits("normal", (n, 1, V), seed=24).clone()
    rng = np.random.default_rng(n)
    for b in range(n):
        if b % 5 == 1:
            x[b, 0, 4000:] = -20.0
        elif b % 5 == 2:
            x[b, 0, :115000] = -20.0
        elif b % 5 == 3:
            x[b, 0, rng.integers(0, V, 4)] = 16.0
        elif b % 5 == 4:
            x[b, 0, 58000:62000] = 9.0            # more equal ones than a CTA's list holds
    s = _settings(n, 30, "m")
    s["min_p"] = (10.0 ** rng.uniform(-4, -0.1, n)).astype(np.float32)
    s["temperature"] = np.ones(n, np.float32)
    u = rng.random((n, 1)).astype(np.float32)
    _check(x, s, u, what="min-p")
    s["top_k"] = rng.choice([0, 100, 255, 256, 257], n).astype(np.int32)
    _check(x, s, u, what="min-p and top-k")


@pytest.mark.parametrize("B,V", [(8, 300), (8, 5003), (90, 12007), (20, 70001)])
def test_settings_outside_their_ranges(B, V):
    """NaN temperature, top_p and min_p; negative ones; min_p above 1; negative
    and huge top_k: each counts as the header says."""
    nan, inf = float("nan"), float("inf")
    x = _logits("peaked", (B, 2, V), seed=V)
    u = np.random.default_rng(V).random((B, 2)).astype(np.float32)

    def full(values, dtype=np.float32):
        return np.resize(np.array(values, dtype), B)

    ones = np.ones(B, np.float32)
    none = dict(top_k=None, top_p=None, min_p=None)
    for name, values in (("top_p", [nan, -0.5, -inf, inf, 1.5, 1e-30, 1e-45]),
                         ("min_p", [nan, -1.0, 1.0, 1.5, inf, -inf, 1e-45, 1e-30])):
        _check(x, {"temperature": ones, **none, name: full(values)}, u, what=name)
    k = full([-1, -2 ** 31, 2 ** 31 - 1, V, V + 1, V - 1, 0], np.int64).astype(np.int32)
    _check(x, {"temperature": ones, **none, "top_k": k}, u, what="top_k")
    T = full([nan, -1.0, -inf, 0.0, -0.0, inf, 1e-45, 1.0])
    t, _, lp = _check(x, {"temperature": T, **none}, u, what="temperature")
    greedy = x[:5].double().argmax(dim=2).numpy()
    assert np.array_equal(t[:5].cpu().numpy(), greedy) and not lp[:5].any()
    _check(x, dict(temperature=T, top_k=k, top_p=full([nan, -0.5, inf, 0.7]),
                   min_p=full([nan, 2.0, -1.0])), u, what="all at once")
