"""The operators of a verify step together, as a serving loop runs them: the
head norms and rotation of a fused projection's rows, the sink attention that
writes and reads the cache, the sampled verification of the drafts, and the
next step from the accepted prefix.  Every stage is checked against its fp64
definition on the inputs the GPU gave it, by the tolerances of its own tests."""
import numpy as np
import pytest
import torch

import oracle.verify_step as vs

pytestmark = pytest.mark.gpu

B, Q, HQ, HKV, D, L, W, S, V, HID = 3, 5, 4, 2, 128, 192, 24, 3, 1200, 96


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sliding_window_speculative_gb300 import build
    build.build()
    yield


def _f64(t):
    return t.to(torch.float64).cpu().numpy()


class Layer:
    """Seeded weights and a cache with its first tokens already in it."""

    def __init__(self, page):
        g = torch.Generator().manual_seed(31)
        rnd = lambda *s: torch.randn(s, generator=g).cuda()  # noqa: E731
        self.w_qkv = (rnd(HID, (HQ + 2 * HKV) * D) / HID ** 0.5).to(torch.bfloat16)
        self.w_out = (rnd(HQ * D, V) / 4).to(torch.bfloat16)
        self.qw, self.kw = 0.5 + torch.rand(D, generator=g).cuda(), 0.5 + torch.rand(D, generator=g).cuda()
        self.f = (10000.0 ** (-torch.arange(D // 2, dtype=torch.float64) * 2 / D)).float().cuda()
        self.temp = torch.tensor([0.0, 0.7, 1.1]).cuda()
        self.top_k = torch.tensor([0, 40, 0], dtype=torch.int32).cuda()
        self.top_p = torch.tensor([1.0, 1.0, 0.9]).cuda()
        self.page = page
        self.table = None
        shape = (B, HKV, L, D)
        if page:
            nb = L // page
            self.table = torch.randperm(B * nb, generator=g).view(B, nb).to(torch.int32).cuda()
            shape = (B * nb, HKV, page, D)
        self.k, self.v = (rnd(*shape).to(torch.bfloat16) for _ in range(2))

    def rows(self, cache, b, n):
        """Positions [0, n) of sequence b, [Hkv, n, D]."""
        if not self.page:
            return cache[b, :, :n]
        j = torch.arange(n, device="cuda")
        return cache[self.table[b].long()[j // self.page], :, j % self.page].transpose(0, 1)

    def step(self, x, pos, draft, u, fused):
        import sliding_window_speculative_gb300 as swa
        qkv = (x @ self.w_qkv).view(B, Q, HQ + 2 * HKV, D)
        q, k, v = qkv.split([HQ, HKV, HKV], dim=2)
        norm = (self.qw, self.kw, 1e-6, self.f)
        lens = pos + Q
        if fused:
            q, k_new, v_new = swa.swa_qk_norm_rope(q, k, v, *norm, pos)
            out, lse = swa.swa_sink_verify_attn(q, self.k, self.v, lens, pos, W, S, D ** -0.5,
                                                k_new=k_new, v_new=v_new, block_table=self.table)
        else:
            q = swa.swa_qk_norm_rope_append(q, k, v, *norm, self.k, self.v, lens, pos,
                                            block_table=self.table)
            out, lse = swa.swa_sink_verify_attn(q, self.k, self.v, lens, pos, W, S, D ** -0.5,
                                                block_table=self.table)
        logits = (out.view(B, Q, HQ * D) @ self.w_out).contiguous()
        toks, acc, lp = swa.swa_sample_accept(logits, u, self.temp, self.top_k, self.top_p,
                                              draft=draft)
        return dict(qkv=qkv, q=q, out=out, lse=lse, logits=logits, tokens=toks, accepted=acc,
                    logprobs=lp)


def _inputs(n_steps, seed=5):
    g = torch.Generator().manual_seed(seed)
    return [dict(x=torch.randn((B, Q, HID), generator=g).to(torch.bfloat16).cuda(),
                 draft=torch.randint(0, V, (B, Q - 1), generator=g).to(torch.int32).cuda(),
                 u=torch.rand((B, Q), generator=g).cuda()) for _ in range(n_steps)]


def _check(layer, r, pos, draft, u):
    pos_h = pos.cpu().numpy().astype(np.int64)
    where = (pos_h[:, None] + np.arange(Q)).reshape(-1)
    qkv = _f64(r["qkv"]).reshape(B * Q, HQ + 2 * HKV, D)
    want, size = vs.norm_rope(qkv[:, :HQ], _f64(layer.qw), 1e-6, _f64(layer.f), where)
    got = _f64(r["q"]).reshape(want.shape)
    assert np.all(np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -18 * size)
    want, size = vs.norm_rope(qkv[:, HQ:HQ + HKV], _f64(layer.kw), 1e-6, _f64(layer.f), where)
    want, size = (a.reshape(B, Q, HKV, D) for a in (want, size))
    for b in range(B):
        n = int(pos_h[b]) + Q
        k, v = _f64(layer.rows(layer.k, b, n)), _f64(layer.rows(layer.v, b, n))
        new = k[:, -Q:].transpose(1, 0, 2)
        assert np.all(np.abs(new - want[b]) <= 2.0 ** -8 * np.abs(want[b]) + 2.0 ** -18 * size[b])
        assert np.array_equal(v[:, -Q:].transpose(1, 0, 2), _f64(r["qkv"][b, :, HQ + HKV:]))
        o, l, absv, mag = vs.sink_attention(_f64(r["q"][b]), k, v, n, int(pos_h[b]), W, S, D ** -0.5)
        d = (D + 8) * 2.0 ** -24 * mag + 2.0 ** -20
        assert np.all(np.abs(_f64(r["out"][b]) - o) <=
                      2.0 ** -8 * np.abs(o) + (2 * d[..., None] + 2.0 ** -14) * absv)
        assert np.all(np.abs(_f64(r["lse"][b]) - l) <= d + 2.0 ** -20 + 2.0 ** -23 * np.abs(l))
    x = _f64(r["logits"])
    toks = np.array([[vs.sample_row(x[b, i], float(u[b, i]), float(layer.temp[b]),
                                    int(layer.top_k[b]), float(layer.top_p[b]))[0]
                      for i in range(Q)] for b in range(B)])
    assert np.array_equal(r["tokens"].cpu().numpy(), toks)
    assert np.array_equal(r["accepted"].cpu().numpy(),
                          vs.accepted_prefix(toks, draft.cpu().numpy()))


@pytest.mark.parametrize("page", [0, 16])
@pytest.mark.parametrize("fused", [False, True])
def test_steps_follow_their_definitions(page, fused):
    layer = Layer(page)
    pos = torch.tensor([0, 2, 90], dtype=torch.int32).cuda()
    for k, step in enumerate(_inputs(4)):
        if k > 0:   # drafts of which some are right: the sampled tokens of a dry run
            dry = layer.step(step["x"], pos, step["draft"], step["u"], fused)
            step["draft"][:, :k] = dry["tokens"][:, :k]
        r = layer.step(step["x"], pos, step["draft"], step["u"], fused)
        torch.cuda.synchronize()
        _check(layer, r, pos, step["draft"], step["u"])
        if k > 0:
            assert int(r["accepted"].min()) >= k
        pos = pos + r["accepted"] + 1


@pytest.mark.parametrize("page", [0, 16])
def test_both_ways_write_the_same_cache(page):
    """Rows handed to the attention call or written ahead of it: the same
    cache bits, and the same tokens here."""
    a, b = Layer(page), Layer(page)
    pos = torch.tensor([1, 40, 130], dtype=torch.int32).cuda()
    for step in _inputs(2, seed=6):
        ra = a.step(step["x"], pos, step["draft"], step["u"], True)
        rb = b.step(step["x"], pos, step["draft"], step["u"], False)
        torch.cuda.synchronize()
        assert torch.equal(a.k, b.k) and torch.equal(a.v, b.v) and torch.equal(ra["q"], rb["q"])
        _check(a, ra, pos, step["draft"], step["u"])
        _check(b, rb, pos, step["draft"], step["u"])
        pos = pos + 2


def test_a_captured_step_replays_on_new_inputs():
    layer, plain = Layer(16), Layer(16)
    first, second = _inputs(2, seed=7)
    pos = torch.tensor([4, 33, 100], dtype=torch.int32).cuda()
    st = {k: v.clone() for k, v in first.items()}
    layer.step(**st, pos=pos, fused=True)          # warm-up outside capture
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = layer.step(**st, pos=pos, fused=True)
    for step, at in ((first, [4, 33, 100]), (second, [6, 38, 101])):
        for k in st:
            st[k].copy_(step[k])
        pos.copy_(torch.tensor(at, dtype=torch.int32))
        graph.replay()
        want = plain.step(**step, pos=pos.clone(), fused=True)
        torch.cuda.synchronize()
        for k in ("q", "out", "lse", "logits", "tokens", "accepted", "logprobs"):
            assert torch.equal(r[k], want[k]), k
        for mine, ref in ((layer.k, plain.k), (layer.v, plain.v)):
            for b in range(B):      # (the captured layer's warm-up wrote the first block too)
                n = int(pos[b]) + Q
                assert torch.equal(layer.rows(mine, b, n), plain.rows(ref, b, n))


def test_largest_batch():
    """65,535 sequences, the most an entry point takes: every one's results are
    those of a batch of three that repeats."""
    import sliding_window_speculative_gb300 as swa
    g = torch.Generator().manual_seed(31)
    B, n, D, L, V = 65535, 3, 64, 16, 37
    rep = lambda t: t.repeat((B // n,) + (1,) * (t.dim() - 1)).cuda()  # noqa: E731
    rnd = lambda *s: torch.randn(s, generator=g).to(torch.bfloat16)  # noqa: E731
    x = rnd(n, 2, 4, D)
    pos, lens = torch.tensor([0, 5, 13], dtype=torch.int32), torch.tensor([2, 7, 15], dtype=torch.int32)
    f = (100.0 ** (-torch.arange(D // 2, dtype=torch.float64) / 32)).float().cuda()
    k, v = rnd(n, 1, L, D), rnd(n, 1, L, D)

    def step(x, k, v, pos, lens):
        q = swa.swa_qk_norm_rope_append(x[:, :, :2], x[:, :, 2:3], x[:, :, 3:], None, None, 1e-6, f,
                                        k, v, lens, pos)
        return (q, k, v) + swa.swa_sink_verify_attn(q, k, v, lens, pos, 4, 2, D ** -0.5)

    small = step(x.cuda(), k.cuda(), v.cuda(), pos.cuda(), lens.cuda())
    large = step(*(rep(t) for t in (x, k, v, pos, lens)))
    torch.cuda.synchronize()
    for i, (a, b) in enumerate(zip(large, small)):
        want = b.repeat((B // n,) + (1,) * (b.dim() - 1))
        if i < 3:
            assert torch.equal(a, want)
        else:  # another plan may serve the larger batch: bf16's half step, twice
            err = (a.double() - want.double()).abs()
            assert (err <= 2.0 ** -7 * want.double().abs() + 2.0 ** -12).all(), i
    logits, u = rnd(n, 2, V), torch.rand((n, 2), generator=g)
    draft, T = torch.tensor([[1], [2], [3]], dtype=torch.int32), torch.tensor([0.7, 1.0, 0.0])
    small = swa.swa_sample_accept(logits.cuda(), u.cuda(), T.cuda(), draft=draft.cuda())
    large = swa.swa_sample_accept(rep(logits), rep(u), rep(T), draft=rep(draft))
    torch.cuda.synchronize()
    for a, b in zip(large, small):
        assert torch.equal(a, b.repeat((B // n,) + (1,) * (b.dim() - 1)))
