"""GPU parity of the sampled verification against its fp64 definition: tokens
and accepted counts bit-exact.

Logprobs, derived: where the token has most of the weight they are log1p of
the rest's share, a quotient of two floats (3 roundings, 2^-24 each) and the
function's own 2 units: within 2^-21 of the value.  Elsewhere the logarithm of
such a quotient: its argument's 2^-22 as an absolute error, and 2 units, on a
value of at least ln 2.  Together within 2^-20 of the value.  To that come
errors that do not shrink with the value: a relative error e of w / S moves
ln(w / S) by e however near 0 that is.  The weights' 2^-39 (numerator and sum)
make 2^-38, the fp64 side's running sum of up to 2^18 terms, 2^-53 each, at
most 2^-35: together below 2^-34."""
import numpy as np
import pytest
import torch

import oracle
import oracle.verify_step as vs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sliding_window_speculative_gb300 import build
    build.build()
    yield


def _logits(kind, shape, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(shape, generator=g) * 2.5
    if kind == "peaked":
        x = x + 12 * (torch.rand(shape, generator=g) < 4.0 / shape[-1])
    elif kind == "ties":
        x = torch.randint(-3, 4, shape, generator=g).float()
    elif kind == "special":     # NaN, -inf and the type's lowest value sprinkled
        m = torch.rand(shape, generator=g)
        x[m < 0.1] = float("nan")
        x[(m >= 0.1) & (m < 0.4)] = float("-inf")
        x[(m >= 0.4) & (m < 0.6)] = torch.finfo(torch.bfloat16).min
    elif kind == "negative":
        x = -x.abs() - 3
    elif kind == "small":       # far below 1, both signs, zeros of both signs
        x = x * 1e-30
        x[torch.rand(shape, generator=g) < 0.1] = 0.0
        x[torch.rand(shape, generator=g) < 0.1] = -0.0
    elif kind == "large":
        x = x * 300
    return x.to(torch.bfloat16)


def _settings(B, seed, mode):
    rng = np.random.default_rng(seed)
    s = dict(temperature=rng.choice([0.5, 0.8, 1.0, 1.7], B), top_k=None, top_p=None, min_p=None)
    if mode in ("k", "all"):
        s["top_k"] = rng.choice([0, 1, 2, 17, 64, 200, 400, 5000], B)
    if mode in ("p", "all"):
        s["top_p"] = rng.choice([0.0, 0.1, 0.5, 0.9, 0.99, 1.0], B)
    if mode in ("m", "all"):
        s["min_p"] = rng.choice([0.0, 0.001, 0.05, 0.3, 1.0], B)
    if mode == "all":
        s["temperature"] = rng.choice([0.0, -1.0, 0.5, 1.0, 3.0], B)
    return {k: None if v is None else v.astype(np.int32 if k == "top_k" else np.float32)
            for k, v in s.items()}


def _row_settings(s, b):
    out = dict(T=float(s["temperature"][b]))
    for k in ("top_k", "top_p", "min_p"):
        if s[k] is not None:
            out[k] = float(s[k][b])
    return out


def _check(x, s, u, draft=None, keep=None, what=""):
    """One call against the definition; tokens, logprobs, accepted."""
    import sliding_window_speculative_gb300 as swa
    B, q_len, V = x.shape
    xs = x.double().numpy()
    cols, lps = np.zeros((B, q_len), np.int64), np.zeros((B, q_len))
    for b in range(B):
        for i in range(q_len):
            cols[b, i], lps[b, i] = vs.sample_row(xs[b, i], float(u[b, i]), **_row_settings(s, b))
    toks = cols if keep is None else keep.numpy()[cols]
    if draft is None and q_len > 1:
        rng = np.random.default_rng(V)
        draft = toks[:, :-1].copy()
        for b in range(B):
            n = rng.integers(0, q_len)
            if n < q_len - 1:
                draft[b, n] += 1
    dev = {k: None if v is None else torch.from_numpy(v).cuda() for k, v in s.items()}
    d = None if q_len == 1 else torch.from_numpy(draft).to(torch.int32).cuda()
    t, acc, lp = swa.swa_sample_accept(x.cuda(), torch.from_numpy(u).cuda(), **dev, draft=d,
                                       keep_ids=None if keep is None else keep.cuda())
    torch.cuda.synchronize()
    assert np.array_equal(t.cpu().numpy(), toks), what
    err = np.abs(lp.double().cpu().numpy() - lps)
    assert np.all(err <= 2.0 ** -20 * np.abs(lps) + 2.0 ** -34), (what, err.max())
    want = vs.accepted_prefix(toks, draft if q_len > 1 else np.zeros((B, 0)))
    assert np.array_equal(acc.cpu().numpy(), want), what
    return t, acc, lp


@pytest.mark.parametrize("mode", ["none", "k", "p", "m", "all"])
@pytest.mark.parametrize("kind", ["normal", "peaked", "ties", "special", "negative", "small",
                                  "large"])
def test_kinds_and_filters(kind, mode):
    B, q_len, V = 12, 3, 5003
    x = _logits(kind, (B, q_len, V), seed=len(kind) * 10 + len(mode))
    u = np.random.default_rng(V).random((B, q_len)).astype(np.float32)
    _check(x, _settings(B, 3, mode), u, what=f"{kind} {mode}")


@pytest.mark.parametrize("B,q_len,V", [
    (1, 1, 1), (2, 3, 2), (3, 2, 7), (1, 4, 8), (5, 5, 13), (2, 2, 255), (200, 1, 1000),
    (3, 64, 501), (2, 2, 32768), (2, 3, 32769), (170, 2, 4097), (1, 8, 50257), (2, 2, 65539),
    (1, 2, 131073), (2, 8, 262144), (1, 3, 262139), (1, 2, 262145), (1, 2, 700001),
])
@pytest.mark.parametrize("mode", ["none", "all"])
def test_sizes(B, q_len, V, mode):
    """Vocabularies around every register, cluster and alignment border (odd
    ones start rows at every 2-byte offset), past what a cluster holds too."""
    x = _logits("peaked" if V > 100 else "ties", (B, q_len, V), seed=V)
    u = np.random.default_rng(V + 1).random((B, q_len)).astype(np.float32)
    _check(x, _settings(B, V, mode), u, what=f"V{V}")


def test_every_candidate_of_a_row_and_its_edges():
    """u at the middle of every candidate's share picks it, in order; u
    outside [0, 1) counts as its border."""
    V = 97
    x = _logits("ties", (1, 1, V), seed=4)
    order = vs.sample_order(x[0, 0].double().numpy())
    w = vs.sample_weights(x[0, 0].double().numpy(), order, 1.3)
    cum = np.cumsum(w)
    u = ((cum - w / 2) / cum[-1]).astype(np.float32)
    xs = x.expand(V, 1, V).contiguous()
    s = dict(temperature=np.full(V, 1.3, np.float32), top_k=None, top_p=None, min_p=None)
    t, _, _ = _check(xs, s, u.reshape(V, 1))
    assert t.cpu().numpy().reshape(-1).tolist() == order.tolist()
    edge = np.array([-1.0, 0.0, 1.0, 5.0, np.inf, np.nan, 1 - 2.0 ** -24], np.float32)
    s = dict(temperature=np.full(7, 1.3, np.float32), top_k=None, top_p=None, min_p=None)
    t, _, _ = _check(xs[:7].contiguous(), s, edge.reshape(7, 1))
    assert t.cpu().numpy().reshape(-1).tolist() == [order[i] for i in (0, 0, -1, -1, -1, 0, -1)]


def test_equal_logits_cut_exactly():
    """Equal weights: every cut-off falls on a whole column."""
    V = 1024
    x = torch.full((8, 1, V), -2.0).to(torch.bfloat16)
    u = np.full((8, 1), 0.5, np.float32)
    s = dict(temperature=np.ones(8, np.float32),
             top_k=np.array([0, 0, 512, 512, 10, 3, 1, 2000], np.int32),
             top_p=np.array([1, 0.5, 1, 0.25, 0.5, 0.5, 0.5, 0.75], np.float32),
             min_p=np.array([0, 0, 0, 1, 0, 1, 0.5, 0], np.float32))
    t, _, lp = _check(x, s, u)
    assert t.cpu().numpy().reshape(-1).tolist() == [512, 256, 256, 64, 2, 1, 0, 384]


@pytest.mark.parametrize("V,parts", [(4096, 1), (90001, 1), (300001, 1)])
def test_values_far_below_the_largest_share_a_bin(V, parts):
    """Values under 2^-32 of the row's largest magnitude share a bin; a draw
    in it still follows value, then column, and zeros of both signs tie."""
    rng = np.random.default_rng(V)
    x = np.zeros(V, np.float32)
    n = 600
    cols = rng.permutation(V)[:n]
    x[:] = -np.inf
    x[cols] = np.where(rng.random(n) < 0.5, 1, -1) * 10.0 ** rng.uniform(-38, -11, n)
    x[cols[:40]] = 0.0
    x[cols[40:60]] = -0.0
    x[cols[60]], x[cols[61]] = 1.0, -3.0
    x = torch.from_numpy(x).to(torch.bfloat16)
    order = vs.sample_order(x.double().numpy())
    w = vs.sample_weights(x.double().numpy(), order, 1.0)
    cum = np.cumsum(w)
    picks = rng.permutation(n)[:64]
    u = ((cum - w / 2) / cum[-1])[picks].astype(np.float32)
    xs = x.view(1, 1, V).expand(4, 16, V).contiguous()
    s = dict(temperature=np.ones(4, np.float32), top_k=None, top_p=None, min_p=None)
    t, _, _ = _check(xs, s, u.reshape(4, 16))
    assert t.cpu().numpy().reshape(-1).tolist() == [int(order[m]) for m in picks]


def test_infinities_and_empty_rows():
    V = 600
    x = _logits("normal", (5, 2, V), seed=9)
    x[0, 0, 5:300:7] = float("inf")
    x[0, 1, 17] = float("inf")
    x[1] = float("-inf")
    x[2] = float("nan")
    x[3, 0] = float("-inf")
    x[3, 0, 77] = torch.finfo(torch.bfloat16).min
    x[4, 1] = torch.finfo(torch.bfloat16).min
    u = np.random.default_rng(1).random((5, 2)).astype(np.float32)
    keep = torch.arange(V, dtype=torch.int32).flip(0).contiguous()
    for mode in ("none", "all"):
        t, _, _ = _check(x, _settings(5, 2, mode), u, keep=keep)
        t = t.cpu().numpy()
        assert t[1].tolist() == t[2].tolist() == [V - 1, V - 1] and t[3, 0] == V - 1 - 77


@pytest.mark.parametrize("T", [1e-38, 1e-6, 1e-3, 50.0, 1e6, 3e38, float("inf")])
def test_extreme_temperatures(T):
    x = _logits("normal", (6, 2, 3001), seed=12)
    u = np.random.default_rng(5).random((6, 2)).astype(np.float32)
    s = dict(temperature=np.full(6, T, np.float32), top_k=None, top_p=None, min_p=None)
    _check(x, s, u)
    s["top_p"] = np.full(6, 0.7, np.float32)
    _check(x, s, u)


def test_greedy_equals_swa_greedy_accept():
    import sliding_window_speculative_gb300 as swa
    x = _logits("ties", (9, 8, 7001), seed=2).cuda()
    draft = torch.randint(0, 7001, (9, 7), dtype=torch.int32, device="cuda")
    am, _ = swa.swa_greedy_accept(x, draft)
    draft[:, :4] = am[:, :4]
    am, acc = swa.swa_greedy_accept(x, draft)
    t, a, lp = swa.swa_sample_accept(x, torch.rand((9, 8), device="cuda"),
                                     torch.zeros(9, device="cuda"), draft=draft)
    torch.cuda.synchronize()
    assert torch.equal(t, am) and torch.equal(a, acc) and torch.all(lp == 0)


def test_shares_follow_the_distribution():
    """4096 draws at evenly spaced u: every token's share is its filtered
    probability to within one draw."""
    import sliding_window_speculative_gb300 as swa
    n, V = 4096, 300
    x = _logits("normal", (1, 1, V), seed=6)
    u = ((torch.arange(n, dtype=torch.float64) + 0.5) / n).float()
    t, _, lp = swa.swa_sample_accept(x.expand(n, 1, V).contiguous().cuda(), u.view(n, 1).cuda(),
                                     torch.full((n,), 0.9, device="cuda"),
                                     top_k=torch.full((n,), 40, dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    order = vs.sample_order(x[0, 0].double().numpy())[:40]
    w = vs.sample_weights(x[0, 0].double().numpy(), order, 0.9)
    p = np.zeros(V)
    p[order] = w / w.sum()
    got = np.bincount(t.cpu().numpy().reshape(-1), minlength=V)
    assert np.all(np.abs(got - n * p) <= 1.0 + 1e-6)


def test_streams_capture_and_prepared_calls():
    """Two overlapping calls (the operator keeps no state), a prepared call
    and a captured graph on new contents."""
    import sliding_window_speculative_gb300 as swa
    xs = [_logits("peaked", (16, 4, 20011), seed=s).cuda() for s in (1, 2)]
    us = [torch.rand((16, 4), device="cuda") for _ in xs]
    T = torch.full((16,), 0.8, device="cuda")
    draft = torch.zeros((16, 3), dtype=torch.int32, device="cuda")
    want = [[t.clone() for t in swa.swa_sample_accept(x, u, T, draft=draft)]
            for x, u in zip(xs, us)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    got = [swa.swa_sample_accept(x, u, T, draft=draft, stream=s)
           for x, u, s in zip(xs, us, streams)]
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert all(torch.equal(a, b) for a, b in zip(g, w))
    call = swa.prepare(swa.swa_sample_accept, xs[0], us[0], T, draft=draft)
    outs = [torch.empty_like(t) for t in want[0]]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        swa.swa_sample_accept(xs[0], us[0], T, draft=draft, tokens=outs[0], accepted=outs[1],
                              logprobs=outs[2])
    xs[0].copy_(xs[1])
    us[0].copy_(us[1])
    got = call()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want[1]))
    assert all(torch.equal(a, b) for a, b in zip(outs, want[1]))


def test_launch_failures_are_reported():
    import sliding_window_speculative_gb300 as swa
    x = _logits("normal", (2, 2, 500), seed=1).cuda()
    u, T = torch.rand((2, 2), device="cuda"), torch.ones(2, device="cuda")
    d = torch.zeros((2, 1), dtype=torch.int32, device="cuda")
    for nth in (1, 2):
        swa.swa_set_debug_options(fail_launch=nth)
        with pytest.raises(swa.SwaError) as e:
            swa.swa_sample_accept(x, u, T, draft=d)
        assert e.value.status == swa.SWA_ERR_CUDA
    assert swa.swa_get_debug_options()["fail_launch"] == 0
    swa.swa_sample_accept(x, u, T, draft=d)
    torch.cuda.synchronize()


def test_offsets_past_32_bits():
    """The last rows of logits with more than 2^31 elements."""
    import sliding_window_speculative_gb300 as swa
    V, rows, last = 262147, 8210, 24
    x = torch.empty((rows, 1, V), dtype=torch.bfloat16, device="cuda")
    x[:-last] = 0
    x[-last:] = _logits("peaked", (last, 1, V), seed=3).cuda()
    u = torch.rand((rows, 1), device="cuda")
    T = torch.full((rows,), 0.9, device="cuda")
    k = torch.zeros(rows, dtype=torch.int32, device="cuda")
    k[:-last] = 1
    k[-last::2] = 50
    t, _, lp = swa.swa_sample_accept(x, u, T, top_k=k)
    want = swa.swa_sample_accept(x[-last:].contiguous(), u[-last:].contiguous(),
                                 T[-last:].contiguous(), top_k=k[-last:].contiguous())
    torch.cuda.synchronize()
    assert torch.equal(t[-last:], want[0])
    assert (lp[-last:] - want[2]).abs().max().item() <= 2.0 ** -19 * want[2].abs().max().item()
    assert not t[:-last].any()


def test_rows_that_outgrow_their_first_chunk():
    """The largest logit far above the first chunk's (the histogram's top is
    raised and the row counted again), or only behind it; lists that overflow
    (equal logits above the bound) fall back to the histogram."""
    V = 70001
    base = _logits("normal", (1, 1, V), seed=21)[0, 0]
    rows = []
    for kind in range(12):
        x = base.clone()
        if kind == 0:
            x[60000:60005] = 3.0e4             # far above 16 times the first chunk's largest
        elif kind == 1:
            x[:40000] = float("-inf")          # nothing in the first chunk
        elif kind == 2:
            x[:40000] = float("nan")
            x[69999] = float("inf")
        elif kind == 3:
            x[:] = 1.5                         # one value everywhere
        elif kind == 4:
            x[:40000] = -300.0                 # negative first, positive behind
        elif kind == 5:
            x[:] = -1.0e30
            x[65000] = -9.0e29
        elif kind == 6:
            x[30000:] = 7.0                    # more columns at the bound than the list holds
        elif kind == 7:
            x[:] = float("-inf")
            x[V - 1] = -5.0
        elif kind == 8:
            x[:40000] = torch.finfo(torch.bfloat16).min   # a masked half, finite
        elif kind == 9:
            x[:40000] = -1.0e6
            x[40000:] *= 1e-3
        elif kind == 10:
            x[:] = -1.0e-12                    # the maximum itself vanishes beside T
        else:
            x[:] = 1.0e-12
            x[5] = -1.0e-12
        rows.append(x)
    n = len(rows)
    xs = torch.stack(rows).view(n, 1, V)
    u = np.random.default_rng(2).random((n, 1)).astype(np.float32)
    for mode in ("none", "k", "p", "m", "all"):
        for T in (0.8, 40.0):
            s = _settings(n, 17, mode)
            s["temperature"] = np.full(n, T, np.float32)
            _check(xs, s, u, what=f"{mode} T{T}")
    # as many rows as make every CTA take a row for itself
    many = xs.repeat(40, 1, 1)
    s = _settings(40 * n, 19, "all")
    _check(many, s, np.random.default_rng(4).random((40 * n, 1)).astype(np.float32), what="one CTA per row")


@pytest.mark.parametrize("n", [2, 30, 70, 160])
def test_lists_of_every_length(n):
    """min-p alone at lines that leave from one to many thousands of columns
    listed: given up after the first chunk, cut by the row's own maximum, sorted
    in each way; rows whose large logits lie in the first chunk only (which
    promises more than there are) or behind it only."""
    V = 150001
    x = _logits("normal", (n, 1, V), seed=23).clone()
    rng = np.random.default_rng(n)
    for b in range(n):
        if b % 5 == 1:
            x[b, 0, 4000:] = -20.0
        elif b % 5 == 2:
            x[b, 0, :140000] = -20.0
        elif b % 5 == 3:
            x[b, 0, rng.integers(0, V, 4)] = 16.0
    s = _settings(n, 29, "m")
    s["min_p"] = (10.0 ** rng.uniform(-4, -0.1, n)).astype(np.float32)
    s["temperature"] = np.full(n, 1.0, np.float32)
    u = rng.random((n, 1)).astype(np.float32)
    _check(x, s, u, what="min-p")
    s["top_k"] = rng.choice([0, 100, 255, 256, 257], n).astype(np.int32)
    _check(x, s, u, what="min-p and top-k")
