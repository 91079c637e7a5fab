"""Token log probabilities against the fp64 definition.

Tokens and ranks are compared as whole numbers.  With y = (x - max) / T, each y
is off by 2^-23 |y| (a difference, a quotient or its product with a rounded
1 / T), the sum of n weights by n' 2^-24 of itself with n' the longest chain of
additions (at most V / 32 + 64) and 2^-21 from an exponential: a log probability
is within 2^-22 (|y| + 1) + (V / 32 + 64) 2^-24 + 2^-20, and the entropy, a
weighted mean of |y| beside the logarithm, within that times (1 + H + the mean |y|)."""
import numpy as np
import pytest
import torch

import oracle.kv8 as kv8

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sliding_window_speculative_gb300 import build
    build.build()
    yield


def check(x, tokens, top=0, T=None, keep=None, rows=None):
    """x bf16 [B, q, V] on the host; every row (or the listed ones) against the
    definition."""
    import sliding_window_speculative_gb300 as swa
    B, q, V = x.shape
    dev = lambda t, dt: None if t is None else torch.as_tensor(np.asarray(t)).to(dt).cuda()  # noqa: E731
    got = swa.swa_token_logprobs(x.cuda(), dev(tokens, torch.int32), top_n=top,
                                 temperature=dev(T, torch.float32), keep_ids=dev(keep, torch.int32))
    torch.cuda.synchronize()
    lp, rank, ent, tt, tl = [None if t is None else t.cpu().numpy() for t in got]
    assert (tt is None) == (top == 0)
    xs = x.double().numpy()
    for b, i in rows or [(b, i) for b in range(B) for i in range(q)]:
        t = 1.0 if T is None else float(np.float32(T[b]))
        w_lp, w_rank, w_ent, w_tt, w_tl = kv8.logprob_row(xs[b, i], tokens[b][i], t, top, keep)
        what = (b, i)
        base = (V / 32 + 64) * 2.0 ** -24 + 2.0 ** -20

        def near(a, w):
            if abs(w) > np.finfo(np.float32).max:     # (what fp32 holds of it)
                return a == np.copysign(np.inf, w)
            # |y| is at most |log probability|: the largest weight is 1
            return abs(a - w) <= 2.0 ** -22 * (abs(w) + 1) + base

        assert near(lp[b, i], w_lp), (what, lp[b, i], w_lp)
        assert rank[b, i] == w_rank, (what, rank[b, i], w_rank)
        assert abs(ent[b, i] - w_ent) <= (base + 2.0 ** -22) * (1 + 2 * w_ent), (what, ent[b, i], w_ent)
        if top:
            assert np.array_equal(tt[b, i], w_tt), (what, tt[b, i], w_tt)
            assert all(near(a, w) for a, w in zip(tl[b, i], w_tl)), what


def logits(B, q, V, seed=0, gain=2.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn((B, q, V), generator=g) * gain).to(torch.bfloat16)


@pytest.mark.parametrize("V", [1, 2, 3, 7, 8, 9, 31, 33, 255, 256, 257, 511, 513, 1000, 2047, 4099,
                               12001])
@pytest.mark.parametrize("top", [0, 1, 5, 20, 32])
def test_sizes(V, top):
    if top > V:
        pytest.skip("more alternatives than columns")
    x = logits(2, 3, V, seed=V)
    rng = np.random.default_rng(V)
    check(x, rng.integers(0, V, (2, 3)), top)


@pytest.mark.parametrize("V", [32768, 50257, 131072, 262144, 262147])
@pytest.mark.parametrize("rows", [(1, 1), (1, 8), (20, 3), (64, 5)])
def test_long_rows(V, rows):
    """Every launch shape: rows that many SMs share, rows of their own."""
    B, q = rows
    x = logits(B, q, V, seed=1)
    rng = np.random.default_rng(2)
    tok = rng.integers(0, V, (B, q))
    for b in range(B):
        tok[b, 0] = int(x[b, 0].float().argmax())
    some = [(0, 0), (B - 1, q - 1), (B // 2, q // 2), (B // 3, 0)]
    check(x, tok, 20, T=np.linspace(0.3, 1.5, B), rows=sorted(set(some)))


@pytest.mark.parametrize("V,top", [(200, 32), (1000, 5), (3001, 20)])
def test_many_short_rows(V, top):
    x = logits(30, 40, V, seed=4)
    tok = np.random.default_rng(1).integers(0, V, (30, 40))
    check(x, tok, top, rows=[(0, 0), (7, 39), (15, 20), (29, 39), (29, 0)])


def test_large_logits_crowded():
    """The largest logits next to one another, so that one warp's columns hold all
    of the first tokens, in rows of either block size."""
    for V in (16000, 120000):
        x = logits(1, 4, V, seed=12)
        x[0, 0, 4096:4352] = 30.0
        x[0, 1, 2048:2304] = torch.arange(256).float().add(20).to(torch.bfloat16)
        for k in range(40):
            x[0, 2, 8192 * (k % 14) // 14 * 8 % V] = 25.0
        x[0, 3] = torch.sort(x[0, 3].float()).values.to(torch.bfloat16)
        check(x, [[4100, 2303, 5, V - 1]], 32)


def test_equal_logits_go_by_column():
    V = 5000
    for x in (torch.zeros((1, 2, V)), torch.full((1, 2, V), -3.0)):
        x = x.to(torch.bfloat16)
        check(x, [[0, V - 1]], 32)
    x = logits(1, 4, V, seed=3, gain=0.01)            # few distinct values
    x[0, 1] = (x[0, 1].float() * 4).round().to(torch.bfloat16)
    x[0, 2, ::2] = -0.0
    x[0, 2, 1::2] = 0.0
    x[0, 3, :] = -1.0
    x[0, 3, [4999, 17, 2048, 255, 256, 257, 511]] = 2.0
    check(x, [[4000, 77, 501, 4999]], 20)


def test_rows_in_order():
    """Rising rows (every column is a new largest one) and falling rows."""
    V = 20000
    up = (torch.arange(V).float() / 64).to(torch.bfloat16)
    x = torch.stack([up, up.flip(0)])[None].contiguous()
    check(x, [[V - 1, 3]], 32)


def test_infinities_and_nan():
    V = 3001
    x = logits(1, 9, V, seed=5)
    inf, nan = float("inf"), float("nan")
    x[0, 0, [5, 1000, 2999]] = inf
    x[0, 1, :] = -inf
    x[0, 2, :] = nan
    x[0, 3, ::3] = nan
    x[0, 4, 1:] = -inf
    x[0, 5, ::2] = -inf
    x[0, 6, [0, 3000]] = nan
    x[0, 6, 7] = inf
    x[0, 7, :] = inf
    x[0, 8, :3000] = -inf
    tok = [[1000, 17, 2, 3, 0, 4, 3000, 100, 0]]
    check(x, tok, 20)
    check(x, tok, 32, T=[0.25])
    check(x, [[4, 18, 7, 5, 1, 5, 6, 3000, 3000]], 0)


def test_rows_of_the_lowest_values():
    """Masks of the type's lowest value, alone and beside -inf, and rows whose
    logits are all far below what others are."""
    V = 1500
    low = torch.finfo(torch.bfloat16).min
    x = torch.full((1, 7, V), low)
    x[0, 1, ::2] = -float("inf")
    x[0, 2, 700] = -3.0
    x[0, 3, :] = -1e35
    x[0, 3, 5] = -2e35
    x[0, 4, 1:] = -float("inf")
    x[0, 5, :9] = -2e30
    x[0, 6, :] = 3e38
    x[0, 6, 3] = low
    x = x.to(torch.bfloat16)
    check(x, [[0, 1, 700, 5, 0, 3, 3]], 20)
    check(x, [[9, 2, 3, 6, 7, 1400, 4]], 5, T=[0.1])


def test_temperatures():
    V = 4000
    x = logits(8, 2, V, seed=6)
    T = [0.0, -1.0, float("nan"), 1e-6, 0.05, 1.0, 8.0, float("inf")]
    rng = np.random.default_rng(0)
    tok = rng.integers(0, V, (8, 2))
    T2 = T[:-1] + [3.0e38]
    check(x, tok, 5, T=T2)
    import sliding_window_speculative_gb300 as swa
    args = x.cuda(), torch.from_numpy(tok).int().cuda()
    a = swa.swa_token_logprobs(*args, temperature=torch.tensor(T).cuda())
    b = swa.swa_token_logprobs(*args, temperature=torch.tensor(T2).cuda())
    assert all(torch.equal(p, q) for p, q in zip(a[:3], b[:3]))


def test_tokens_that_are_no_columns():
    V = 700
    x = logits(1, 6, V, seed=7)
    check(x, [[-1, V, V + 5, 2 ** 31 - 1, -2 ** 31, V - 1]], 3)


@pytest.mark.parametrize("V", [1, 300, 12001])
def test_keep_set(V):
    rng = np.random.default_rng(8)
    keep = rng.permutation(4 * V)[:V].astype(np.int32)
    x = logits(3, 4, V, seed=8)
    tok = keep[rng.integers(0, V, (3, 4))]
    tok[0, 0], tok[1, 1] = -1, 4 * V + 3
    absent = np.setdiff1d(np.arange(4 * V), keep)
    if absent.size:
        tok[2, 2] = absent[0]
    check(x, tok, min(V, 7), keep=keep)
    keep[V // 2] = keep[0]                            # the same token twice
    tok[0, 1] = keep[0]
    keep[V - 1] = -7                                  # a column without a token
    tok[0, 2] = -7
    check(x, tok, min(V, 7), keep=keep)


def test_unaligned_rows():
    """Rows that begin at any 2-byte address, of a tensor that does."""
    import sliding_window_speculative_gb300 as swa
    for V in (1023, 4097):
        for off in range(9):
            flat = logits(1, 1, 3 * V + off, seed=off).view(-1)
            x = flat[off:].view(1, 3, V)
            base = torch.empty(3 * V + 16, dtype=torch.bfloat16, device="cuda")
            view = base[off:off + 3 * V]
            view.copy_(x.reshape(-1))
            tok = torch.tensor([[0, V // 2, V - 1]], dtype=torch.int32, device="cuda")
            got = swa.swa_token_logprobs(view.view(1, 3, V), tok, top_n=4)
            want = swa.swa_token_logprobs(x.contiguous().cuda(), tok, top_n=4)
            for a, b in zip(got, want):
                assert torch.equal(a, b) if a.dtype == torch.int32 else torch.allclose(
                    a, b, rtol=0, atol=1e-4)


def test_the_same_results_every_time():
    import sliding_window_speculative_gb300 as swa
    x = logits(16, 8, 50257, seed=9).cuda()
    tok = torch.randint(0, 50257, (16, 8), dtype=torch.int32).cuda()
    first = swa.swa_token_logprobs(x, tok, top_n=20)
    for _ in range(3):
        again = swa.swa_token_logprobs(x, tok, top_n=20)
        assert all(torch.equal(a, b) for a, b in zip(first, again))


def test_offsets_past_32_bits():
    """More than 2^32 bytes of logits."""
    import sliding_window_speculative_gb300 as swa
    B, q, V = 20, 512, 262144
    x = torch.zeros((B, q, V), dtype=torch.bfloat16, device="cuda")
    x[B - 1, q - 1, V - 3] = 5.0
    tok = torch.full((B, q), V - 3, dtype=torch.int32, device="cuda")
    lp, rank, ent, tt, tl = swa.swa_token_logprobs(x, tok, top_n=2)
    assert rank[B - 1, q - 1].item() == 1 and tt[B - 1, q - 1].tolist() == [V - 3, 0]
    assert rank[0, 0].item() == V - 2 and tt[0, 0].tolist() == [0, 1]
    z = np.log(V - 1 + np.exp(5.0))
    assert abs(lp[B - 1, q - 1].item() - (5 - z)) < 1e-3 and abs(lp[0, 0].item() + np.log(V)) < 1e-3
    assert abs(ent[0, 0].item() - np.log(V)) < 1e-2


def test_given_outputs_and_refusals():
    import sliding_window_speculative_gb300 as swa
    x = logits(2, 3, 100).cuda()
    tok = torch.zeros((2, 3), dtype=torch.int32, device="cuda")
    lp = torch.empty((2, 3), device="cuda")
    got = swa.swa_token_logprobs(x, tok, logprobs=lp)
    assert got[0] is lp and got[3] is None and got[4] is None
    bad = [dict(top_n=33), dict(top_n=-1), dict(tokens=tok.long()), dict(tokens=tok[:1]),
           dict(logits=x.float()), dict(logits=x[0]), dict(temperature=torch.ones(3).cuda()),
           dict(keep_ids=torch.zeros(99, dtype=torch.int32).cuda()), dict(ranks=lp),
           dict(top_tokens=tok), dict(tokens=None), dict(entropy=lp[:1])]
    for over in bad:
        kw = {"logits": x, "tokens": tok, **over}
        with pytest.raises((TypeError, ValueError, swa.SwaError)):
            swa.swa_token_logprobs(**kw)
            pytest.fail(f"{over} was taken")
    short = logits(1, 1, 5).cuda()
    with pytest.raises(ValueError):
        swa.swa_token_logprobs(short, tok[:1, :1], top_n=6)
