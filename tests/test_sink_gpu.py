"""GPU parity of the sink attention against its fp64 definition, on every
kernel, contiguous and paged caches, with and without the fused append.

Every cache row that no query of its sequence sees holds NaN, so a read that
reaches a result shows.

Tolerance, derived: scores are sums of D products of bf16 values (exact in
fp32) and one scaling, in fp32: off by at most (D + 8) 2^-24 of their summed
magnitude `mag`; exponents and running sums add below 2^-20.  With d the sum
of both, a weight is off by d relative (weights are carried to 2^-16 besides),
so an output by (2 d + 2^-14) of the weighted |v|, and by the one rounding to
bf16, 2^-8 of itself; lse by d, its logarithm by 2^-20 and its fp32 rounding."""
import numpy as np
import pytest
import torch

import oracle.verify_step as vs
from tests.helpers import forced_kernel

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sliding_window_speculative_gb300 import build
    build.build()
    yield


@pytest.fixture(params=["plan", "simt", "tc", "rows"])
def kernel(request):
    with forced_kernel(request.param):
        yield request.param


class Case:
    """One batch: q, caches with NaN where nothing looks, positions."""

    def __init__(self, q_len, Hq, Hkv, D, W, S, pos, L, lens=None, page=0, append=False, seed=0):
        B = len(pos)
        g = torch.Generator().manual_seed(seed + q_len + D + W + S)
        rnd = lambda *s: torch.randn(s, generator=g).to(torch.bfloat16)  # noqa: E731
        lens = [p + q_len for p in pos] if lens is None else lens
        self.W, self.S, self.D, self.page, self.L = W, S, D, page, L
        self.pos, self.lens, self.scale = pos, lens, D ** -0.5
        self.q = rnd(B, q_len, Hq, D)
        self.k, self.v = rnd(B, Hkv, L, D), rnd(B, Hkv, L, D)
        self.k[torch.rand(self.k.shape, generator=g) < 0.01] *= 8
        seen = torch.zeros(B, L, dtype=torch.bool)
        for b in range(B):
            for i in range(q_len):
                p = pos[b] + i
                hi = max(0, min(p + 1, lens[b], L))
                seen[b, max(0, p - W + 1):hi] = True
                seen[b, :min(S, hi)] = True
        for c in (self.k, self.v):
            c.masked_fill_(~seen[:, None, :, None], float("nan"))
        self.new = None
        if append:
            self.new = []
            for c in (self.k, self.v):
                rows = rnd(B, q_len, Hkv, D)
                for b in range(B):
                    for i in range(q_len):
                        j = pos[b] + i
                        if j < min(lens[b], L):
                            rows[b, i] = c[b, :, j]
                self.new.append(rows)

    def reference(self):
        f = lambda t: t.double().numpy()  # noqa: E731
        per = [vs.sink_attention(f(self.q[b]), np.nan_to_num(f(self.k[b])), np.nan_to_num(f(self.v[b])),
                                 self.lens[b], self.pos[b], self.W, self.S, self.scale)
               for b in range(len(self.pos))]
        return [np.stack(x) for x in zip(*per)]

    def device(self, seed=0):
        """(k_cache, v_cache, block_table, k_new, v_new) on the GPU; new rows
        of an append are NaN in the cache."""
        k, v = self.k.clone(), self.v.clone()
        if self.new is not None:
            for b, p in enumerate(self.pos):
                k[b, :, p:p + self.q.shape[1]] = v[b, :, p:p + self.q.shape[1]] = float("nan")
        table = None
        if self.page:
            B, Hkv, L, D = k.shape
            nb = L // self.page
            g = torch.Generator().manual_seed(seed)
            table = torch.randperm(B * nb + 2, generator=g)[:B * nb].view(B, nb).to(torch.int32)
            pools = []
            for c in (k, v):
                pool = torch.full((B * nb + 2, Hkv, self.page, D), float("nan"), dtype=c.dtype)
                pool[table.view(-1).long()] = c.view(B, Hkv, nb, self.page, D).transpose(1, 2).reshape(
                    B * nb, Hkv, self.page, D)
                pools.append(pool)
            k, v = pools
            table = table.cuda()
        new = [None, None] if self.new is None else [t.cuda() for t in self.new]
        return k.cuda(), v.cuda(), table, new[0], new[1]

    def run(self, splits=0):
        import sliding_window_speculative_gb300 as swa
        k, v, table, kn, vn = self.device()
        i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
        out, lse = swa.swa_sink_verify_attn(self.q.cuda(), k, v, i32(self.lens), i32(self.pos), self.W,
                                            self.S, self.scale, k_new=kn, v_new=vn,
                                            block_table=table, num_splits=splits)
        torch.cuda.synchronize()
        assert swa.swa_read_device_errors() == 0
        if self.new is not None:
            self.check_cache(k, v, table)
        return out, lse

    def check_cache(self, k, v, table):
        """Exactly the new rows were written."""
        k0, v0, _, kn, vn = self.device()
        for b, p in enumerate(self.pos):
            for i in range(self.q.shape[1]):
                j = p + i
                if j >= min(self.lens[b], self.L):
                    continue
                if table is None:
                    k0[b, :, j], v0[b, :, j] = kn[b, i], vn[b, i]
                else:
                    at = (int(table[b, j // self.page]), slice(None), j % self.page)
                    k0[at], v0[at] = kn[b, i], vn[b, i]
        for got, want in ((k, k0), (v, v0)):
            assert torch.equal(got.view(torch.int16), want.view(torch.int16))

    def check(self, out, lse, what):
        o, l, absv, mag = self.reference()
        got, gl = out.double().cpu().numpy(), lse.double().cpu().numpy()
        assert np.all(np.isfinite(got)), what
        d = (self.D + 8) * 2.0 ** -24 * mag + 2.0 ** -20
        tol = 2.0 ** -8 * np.abs(o) + (2 * d[..., None] + 2.0 ** -14) * absv
        err = np.abs(got - o)
        assert np.all(err <= tol), (what, (err - tol).max())
        fin = np.isfinite(l)
        assert np.array_equal(fin, np.isfinite(gl)), what
        assert np.all(gl[~fin] == -np.inf) and np.all(got[~fin] == 0), what
        lerr = np.abs(gl[fin] - l[fin])
        assert np.all(lerr <= d[fin] + 2.0 ** -20 + 2.0 ** -23 * np.abs(l[fin])), (what, lerr.max())


POS = [0, 1, 5, 11, 30, 37, 64, 100, 201, 300]


@pytest.mark.parametrize("S", [1, 4, 8, 13, 127, 128])
@pytest.mark.parametrize("D,q_len", [(256, 8), (128, 8), (64, 3), (256, 1), (128, 40), (256, 33)])
def test_contiguous(kernel, D, q_len, S):
    c = Case(q_len, 8, 2, D, 37, S, POS, 384, seed=1)
    c.check(*c.run(), f"{kernel} D{D} q{q_len} S{S}")


@pytest.mark.parametrize("W", [1, 7, 188])
@pytest.mark.parametrize("page", [8, 24, 64])
@pytest.mark.parametrize("S", [3, 16, 77])
def test_paged(kernel, page, W, S):
    c = Case(8, 8, 2, 128, W, S, POS, 384, page=page, seed=2)
    c.check(*c.run(), f"{kernel} page {page} W{W} S{S}")


@pytest.mark.parametrize("W,S", [(5, 4), (37, 1), (37, 30), (1, 9), (100, 128)])
@pytest.mark.parametrize("page", [0, 8, 24])
@pytest.mark.parametrize("D,q_len", [(256, 8), (128, 40), (64, 9), (128, 1)])
def test_fused_append(kernel, D, q_len, page, W, S):
    """The block's own rows among the sinks, in the window, and both."""
    c = Case(q_len, 4, 2, D, W, S, POS, 384, page=page, append=True, seed=3)
    c.check(*c.run(), f"{kernel} append D{D} q{q_len} page {page} W{W} S{S}")


@pytest.mark.parametrize("splits", [2, 5, 13, 64])
@pytest.mark.parametrize("page,append", [(0, False), (16, False), (16, True), (0, True)])
def test_split_keys(kernel, splits, page, append):
    c = Case(8, 8, 2, 128, 300, 21, [0, 3, 40, 318, 400, 900], 1024, page=page, append=append, seed=4)
    c.check(*c.run(splits), f"{kernel} splits {splits} page {page} append {append}")


@pytest.mark.parametrize("S", [1, 100])
def test_prefill_chunks(kernel, S):
    """512-row chunks: early row tiles see the sinks inside their window, late
    ones behind it; the first chunk writes its own sinks."""
    for append in (False, True):
        c = Case(512, 2, 1, 128, 60, S, [0, 3, 700], 1280, append=append, seed=5)
        c.check(*c.run(), f"{kernel} prefill S{S} append {append}")


def test_many_query_heads_and_long_blocks(kernel):
    for Hq, Hkv, q_len, D in ((64, 1, 2, 128), (12, 4, 64, 256), (3, 3, 64, 128), (16, 1, 17, 64)):
        c = Case(q_len, Hq, Hkv, D, 50, 5, [7, 49, 120], 256, seed=6)
        c.check(*c.run(), f"{kernel} {Hq}/{Hkv} q{q_len} D{D}")


def test_large_batch_runs_many_items_per_cta(kernel):
    rng = np.random.default_rng(3)
    for page, append in ((0, False), (16, True)):
        pos = [int(x) for x in rng.integers(0, 180, 170)]
        c = Case(4, 8, 2, 128, 40, 6, pos, 192, page=page, append=append, seed=7)
        c.check(*c.run(), f"{kernel} batch 170 page {page}")


def test_lengths_that_break_the_preconditions(kernel):
    """Sequences shorter than their block, or empty: rows without a visible
    key give 0 and -inf, and nothing outside is read."""
    pos, lens = [0, 10, 100, 50, 250], [0, 3, 100, 52, 300]
    c = Case(8, 8, 2, 128, 20, 6, pos, 256, lens=lens, seed=8)
    c.check(*c.run(), f"{kernel} short lengths")


def test_no_sinks_is_the_windowed_call(kernel):
    import sliding_window_speculative_gb300 as swa
    c = Case(8, 8, 2, 256, 37, 0, POS, 384, seed=9)
    k, v, _, _, _ = c.device()
    i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
    a = swa.swa_sink_verify_attn(c.q.cuda(), k, v, i32(c.lens), i32(c.pos), c.W, 0, c.scale)
    b = swa.swa_verify_attn(c.q.cuda(), k, v, i32(c.lens), i32(c.pos), c.W, c.scale)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("S", [1, 4, 40])
@pytest.mark.parametrize("page,splits", [(0, 0), (8, 0), (0, 4), (16, 3)])
def test_count_probe(kernel, S, page, splits):
    """K = 0: lse is ln of the number of visible keys, so every key counts
    exactly once."""
    c = Case(8, 8, 2, 128, 45, S, [0, 20, 41, 45, 50, 60, 85, 200], 256, page=page, seed=10)
    c.k = torch.where(torch.isnan(c.k), c.k, torch.zeros_like(c.k))
    _, lse = c.run(splits)
    for b, p0 in enumerate(c.pos):
        for i in range(8):
            p = p0 + i
            n = len([j for j in range(p + 1) if j > p - c.W or j < S])
            err = (lse[b, i].double().cpu() - np.log(n)).abs().max().item()
            assert err < 0.25 / n / n + 1e-6, (b, i, n, err)


def test_pinned_pages_in_front_of_a_ring():
    """A ring of window pages with pinned pages for the sinks: the table lists
    the pinned pages first, then the ring over and over."""
    import sliding_window_speculative_gb300 as swa
    W, S, q_len, page, L = 60, 10, 8, 8, 1024
    pinned, ring = 2, 10                       # pages per sequence; 80 >= W + q_len - 1 + 7
    pos = [100, 555, 1000]
    c = Case(q_len, 8, 2, 128, W, S, pos, L, seed=11)
    B, Hkv, _, D = c.k.shape
    per = pinned + ring
    table = torch.tensor([[b * per + (n if n < pinned else pinned + n % ring) for n in range(L // page)]
                          for b in range(B)], dtype=torch.int32)
    pools = []
    for src in (c.k, c.v):
        pool = torch.full((B * per, Hkv, page, D), float("nan"), dtype=torch.bfloat16)
        for b in range(B):
            for j in range(c.lens[b]):
                if j < S or j > pos[b] - W:
                    pool[table[b, j // page], :, j % page] = src[b, :, j]
        pools.append(pool.cuda())
    i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
    out, lse = swa.swa_sink_verify_attn(c.q.cuda(), *pools, i32(c.lens), i32(pos), W, S, c.scale,
                                        block_table=table.cuda())
    torch.cuda.synchronize()
    c.check(out, lse, "ring with pinned pages")


def test_captured_split_plan_and_prepared_call():
    import sliding_window_speculative_gb300 as swa
    cs = [Case(8, 8, 2, 256, 300, 5, [400, 700], 1024, seed=s) for s in (1, 2)]
    i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
    q, (k, v, _, _, _) = cs[0].q.cuda(), cs[0].device()
    sl, qp = i32(cs[0].lens), i32(cs[0].pos)
    args = (q, k, v, sl, qp, 300, 5, cs[0].scale)
    out, lse = swa.swa_sink_verify_attn(*args, num_splits=4)   # grows the workspace
    cs[0].check(out, lse, "split call")
    graph = torch.cuda.CUDAGraph()
    go, gl = torch.empty_like(out), torch.empty_like(lse)
    with torch.cuda.graph(graph):
        swa.swa_sink_verify_attn(*args, out=go, lse=gl, num_splits=4)
    call = swa.prepare(swa.swa_sink_verify_attn, *args, num_splits=4)
    k2, v2, _, _, _ = cs[1].device()
    q.copy_(cs[1].q)
    k.copy_(k2)
    v.copy_(v2)
    a = call()
    cs[1].check(*a, "prepared")
    graph.replay()
    torch.cuda.synchronize()
    cs[1].check(go, gl, "captured")


def test_a_captured_split_survives_a_larger_call():
    """The split workspace grows while a graph that uses the old one lives:
    the replay still finds its own."""
    import sliding_window_speculative_gb300 as swa
    swa.swa_release_workspace()
    small = Case(4, 8, 2, 128, 200, 5, [300], 512, seed=12)
    big = Case(8, 8, 2, 256, 300, 5, [400, 700, 500, 650], 1024, seed=13)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
    k, v, _, _, _ = small.device()
    args = (small.q.cuda(), k, v, i32(small.lens), i32(small.pos), 200, 5, small.scale)
    swa.swa_sink_verify_attn(*args, num_splits=2)
    out, lse = torch.empty_like(small.q).cuda(), torch.empty((1, 4, 8)).cuda()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        swa.swa_sink_verify_attn(*args, out=out, lse=lse, num_splits=2)
    big.check(*big.run(8), "the larger call")
    filler = torch.full((1 << 22,), 3.0e4, device="cuda")   # whatever is free now is overwritten
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    small.check(out, lse, "the captured call")
    del graph, filler
    swa.swa_release_workspace()


def test_offsets_past_32_bits():
    """A cache of more than 2^31 elements: the last rows are attended and
    written where they are."""
    import sliding_window_speculative_gb300 as swa
    D, q_len, W, S = 256, 8, 40, 4
    L = (1 << 31) // D + 4096
    small = Case(q_len, 8, 1, D, W, S, [300], 512, append=True, seed=14)
    p0 = L - q_len - 100
    shift = p0 - 300
    caches = []
    for src in small.device()[:2]:
        c = torch.empty((1, 1, L, D), dtype=torch.bfloat16, device="cuda")
        c[:, :, :S] = src[:, :, :S]
        lo = 300 - W + 1
        c[:, :, lo + shift:300 + shift] = src[:, :, lo:300]
        caches.append(c)
    _, _, _, kn, vn = small.device()
    i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
    for kernel in ("plan", "simt", "rows"):
        with forced_kernel(kernel):
            out, lse = swa.swa_sink_verify_attn(small.q.cuda(), *caches, i32([p0 + q_len]), i32([p0]),
                                                W, S, small.scale, k_new=kn, v_new=vn)
            torch.cuda.synchronize()
        small.check(out, lse, f"far rows, {kernel}")
        for c, n in zip(caches, (kn, vn)):
            assert torch.equal(c[0, :, p0:p0 + q_len].transpose(0, 1), n[0])
