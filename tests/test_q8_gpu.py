"""The 8-bit KV cache on the GPU against its fp64 definition: rows written,
rows read back, and the windowed attention over them.

Written and read rows are compared bit for bit.  Attention, per output, with
u = 2^-24, w_j the row's weights and s_j = scale q.k_j:
  a score      products of a bf16 and an e4m3 number are exact in fp32; D of
               them summed in fp32, scaled by three rounded factors:
               d = (D + 16) u scale sum |q||k| (+ 2^-20 for the exponential),
               which also covers what a query row split into two e4m3 numbers
               loses (2^-22 of its largest element, per element)
  a weight     e^d off, then rounded to 8 bits or more (bf16 over rows read back;
               straight from the cache 11, in three e4m3 numbers: 2^-8 covers both),
               or, where that is more, by 2^-21 of the largest w_j |v_j|'s scale
               (the smallest step of the three numbers): n keys add n 2^-21 of it
  the result   rounded to bf16: 2^-8 of itself
  lse          d + 2^-20, 2^-22 of itself
The largest w_j 448 2^e_j is at most 2 max w_j max|v_j|."""
import numpy as np
import pytest
import torch

import oracle.kv8 as kv8
from tests.helpers import forced_kernel

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sliding_window_speculative_gb300 import build
    build.build()
    yield


E4M3 = torch.float8_e4m3fn


class Cache:
    """A contiguous or paged 8-bit cache of rows at given positions, on the
    host (codes [B, Hkv, L, D], exponents) and on the device."""

    def __init__(self, B, Hkv, L, D, page=0, seed=0, spread=1):
        self.B, self.Hkv, self.L, self.D, self.page = B, Hkv, L, D, page
        rng = np.random.default_rng(seed)
        self.codes, self.exps = [], []
        for _ in range(2):
            c = rng.integers(0, 256, (B, Hkv, L, D)).astype(np.uint8)
            # normally distributed values, a row's largest near 448
            x = rng.standard_normal((B, Hkv, L, D)) * 110
            t = torch.from_numpy(np.clip(x, -448, 448)).float().to(E4M3).view(torch.uint8).numpy()
            c[:] = t
            self.codes.append(c)
            self.exps.append(rng.integers(-8 - spread, -8 + spread + 1, (B, Hkv, L)).astype(np.int8))
        self.table = None
        if page:
            nb = L // page
            self.table = rng.permutation(B * nb + 2)[:B * nb].reshape(B, nb).astype(np.int32)

    def poison(self, seen):
        """NaN elements and wild exponents where seen [B, L] is false."""
        for kv in range(2):
            self.codes[kv] = np.where(seen[:, None, :, None], self.codes[kv], 0x7f).astype(np.uint8)
            wild = np.where(np.arange(self.L) % 2 == 0, 127, -128)
            self.exps[kv] = np.where(seen[:, None, :], self.exps[kv], wild).astype(np.int8)

    def values(self, kv):
        return kv8.row_values(self.codes[kv], self.exps[kv])

    def device(self):
        out = []
        for a in (*self.codes, *self.exps):
            if self.page:
                nb = self.L // self.page
                pool = np.full((self.B * nb + 2, self.Hkv, self.page) + a.shape[3:], 0x7f, a.dtype)
                for b in range(self.B):
                    for k in range(nb):
                        pool[self.table[b, k]] = a[b, :, k * self.page:(k + 1) * self.page]
                a = pool
            out.append(torch.from_numpy(np.ascontiguousarray(a)).cuda())
        self.dev = [out[0].view(E4M3), out[1].view(E4M3), out[2], out[3]]
        self.dev_table = None if self.table is None else torch.from_numpy(self.table).cuda()
        return self.dev

    def host(self):
        """The device's codes and exponents in position order."""
        got = []
        for t in self.dev:
            a = (t.view(torch.uint8) if t.dtype == E4M3 else t).cpu().numpy()
            if self.page:
                nb = self.L // self.page
                flat = np.empty((self.B, self.Hkv, self.L) + a.shape[3:], a.dtype)
                for b in range(self.B):
                    for k in range(nb):
                        flat[b, :, k * self.page:(k + 1) * self.page] = a[self.table[b, k]]
                a = flat
            got.append(a)
        return got


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------ append

def _special_rows(D):
    """Rows of every magnitude, with ties, zeros, infinities and NaN."""
    rng = np.random.default_rng(1)
    rows = [rng.standard_normal(D) * s for s in (1, 1e-3, 300, 1e-14, 1e-18, 1e-30, 1e16, 1e30)]
    rows += [np.zeros(D), np.full(D, -0.0)]
    # every e4m3 value, the middles between neighbours (ties) and a bit past them
    steps = kv8.E4M3[:127]
    for f in (0.5, 0.502, 0.498):
        rows.append(np.resize(steps[:-1] + f * np.diff(steps), D))
    rows.append(np.resize(-steps, D))
    # largest elements around 448 2^k
    for top in (1.75, 1.7578125, 1.7421875, 1.0, 1.9921875):
        r = rng.standard_normal(D) * 0.1
        r[D // 3] = -top * 2.0 ** 5
        rows.append(r)
    r = rng.standard_normal(D)
    r[[0, 5, D - 1]] = [np.inf, np.nan, -np.inf]
    rows.append(r)
    rows.append(np.full(D, np.nan))
    return torch.from_numpy(np.stack(rows)).to(torch.bfloat16)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("page", [0, 8])
def test_append_writes_the_defined_rows(D, page):
    import sliding_window_speculative_gb300 as swa
    rows = _special_rows(D)
    q_len, Hkv, B = 3, 2, -(-len(rows) // 6)
    x = torch.zeros((B * q_len * Hkv, D), dtype=torch.bfloat16)
    x[:len(rows)] = rows
    k = x.view(B, q_len, Hkv, D)
    v = x.flip(0).view(B, q_len, Hkv, D)
    cache = Cache(B, Hkv, 24, D, page)
    cache.device()
    q_pos = [(7 * b) % 21 for b in range(B)]
    lens = [p + 3 for p in q_pos]
    res = swa.swa_q8_append(k.cuda(), v.cuda(), *cache.dev, i32(lens), i32(q_pos),
                            block_table=cache.dev_table)
    torch.cuda.synchronize()
    assert all(a is b for a, b in zip(res, cache.dev))
    want = [c.copy() for c in (*cache.codes, *cache.exps)]
    for kv, t in enumerate((k, v)):
        for b in range(B):
            for i in range(q_len):
                for h in range(Hkv):
                    c, e = kv8.quantise_row(t[b, i, h].double().numpy())
                    want[kv][b, h, q_pos[b] + i], want[2 + kv][b, h, q_pos[b] + i] = c, e
    got = cache.host()
    for g, w in zip(got[:2], want[:2]):
        nan = (w & 127) == 127
        assert np.array_equal(g[~nan], w[~nan]) and np.all((g[nan] & 127) == 127)
    for g, w in zip(got[2:], want[2:]):
        assert np.array_equal(g, w)


def test_append_drops_rows_without_a_place():
    """Rows before position 0, past the sequence's or the cache's end are
    dropped; strided views; no other byte changes."""
    import sliding_window_speculative_gb300 as swa
    B, q_len, Hkv, D, L = 6, 5, 3, 64, 32
    cache = Cache(B, Hkv, L, D)
    cache.device()
    q_pos = [-2, 0, 10, 29, 40, -9]
    lens = [32, 3, 10, 40, 50, 32]
    g = torch.Generator().manual_seed(2)
    qkv = torch.randn((B, q_len, 5 + 2 * Hkv, D), generator=g).to(torch.bfloat16)
    dev = qkv.cuda()
    _, k, v = dev.split([5, Hkv, Hkv], dim=2)
    swa.swa_q8_append(k, v, *cache.dev, i32(lens), i32(q_pos))
    torch.cuda.synchronize()
    want = [c.copy() for c in (*cache.codes, *cache.exps)]
    for kv in range(2):
        for b in range(B):
            for i in range(q_len):
                p = q_pos[b] + i
                if 0 <= p < min(lens[b], L):
                    for h in range(Hkv):
                        row = qkv[b, i, 5 + kv * Hkv + h].double().numpy()
                        want[kv][b, h, p], want[2 + kv][b, h, p] = kv8.quantise_row(row)
    for a, w in zip(cache.host(), want):
        assert np.array_equal(a, w)


@pytest.mark.parametrize("B,q_len,Hkv,D,page", [(1, 1, 1, 64, 0), (300, 3, 5, 128, 16),
                                                (40, 129, 2, 256, 24), (1, 512, 8, 64, 0)])
def test_append_of_many_rows(B, q_len, Hkv, D, page):
    """Against the read back: nearest values of the rows written."""
    import sliding_window_speculative_gb300 as swa
    L = -(-(q_len + 20) // 24) * 48
    cache = [torch.zeros((B * (L // page), Hkv, page, D) if page else (B, Hkv, L, D),
                         dtype=torch.uint8, device="cuda").view(E4M3) for _ in range(2)]
    cache += [torch.zeros(cache[0].shape[:3], dtype=torch.int8, device="cuda") for _ in range(2)]
    table = None
    if page:
        table = torch.randperm(B * (L // page), device="cuda").to(torch.int32).view(B, -1).contiguous()
    g = torch.Generator(device="cuda").manual_seed(5)
    k, v = (torch.randn((B, q_len, Hkv, D), generator=g, device="cuda", dtype=torch.bfloat16)
            for _ in range(2))
    q_pos = torch.randint(0, L - q_len + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
    swa.swa_q8_append(k, v, *cache, q_pos + q_len, q_pos, block_table=table)
    got = swa.swa_q8_read(*cache, q_pos + q_len, q_pos - 1, q_len + 2, block_table=table)
    for x, y in zip((k, v), got):
        y = y.transpose(1, 2).double()
        assert not y[:, 0].any() and not y[:, -1].any()
        x, y = x.double(), y[:, 1:-1]
        top = x.abs().amax(dim=-1, keepdim=True)
        e = torch.ceil(torch.log2(top / 448))
        # (a tie is off by exactly the bound, which pow may give an ulp too low)
        step = 2.0 ** (e - 10) * (1 + 2.0 ** -40)
        assert ((y - x).abs() <= torch.maximum(2.0 ** -4 * x.abs(), step)).all()
        assert ((y - x).abs() > 0).any()


# -------------------------------------------------------------------- read

@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("page", [0, 24])
def test_read_gives_the_rows_or_zeros(D, page):
    import sliding_window_speculative_gb300 as swa
    B, Hkv, L, n = 5, 3, 72, 31
    cache = Cache(B, Hkv, L, D, page, spread=40)
    cache.device()
    lens, start = [72, 40, 0, 9, 200], [41, 20, 0, -15, 60]
    k, v = swa.swa_q8_read(*cache.dev, i32(lens), i32(start), n, block_table=cache.dev_table)
    torch.cuda.synchronize()
    for kv, t in enumerate((k, v)):
        want = np.zeros((B, Hkv, n, D))
        val = cache.values(kv)
        for b in range(B):
            for r in range(n):
                p = start[b] + r
                if 0 <= p < min(lens[b], L):
                    want[b, :, r] = val[b, :, p]
        assert np.array_equal(t.double().cpu().numpy(), want)


def test_read_of_extreme_exponents():
    """Exponents an append never writes: the product is rounded to bf16."""
    import sliding_window_speculative_gb300 as swa
    cache = Cache(1, 1, 8, 64)
    cache.exps = [np.array([[[127, -128, 100, -100, 0, 120, -126, -127]]], np.int8)] * 2
    cache.device()
    k, _ = swa.swa_q8_read(*cache.dev, i32([8]), i32([0]), 8)
    val = torch.from_numpy(cache.values(0)).float()
    ok = torch.from_numpy(np.abs(cache.exps[0].astype(int)) < 121)
    assert torch.equal(k.cpu()[ok], val[ok].to(torch.bfloat16))


# --------------------------------------------------------------- attention

def _attend(B, q_len, Hq, Hkv, D, W, L, lens, q_pos, page=0, splits=0, scale=None, seed=0, spread=1,
            poison=True, q_gain=1.0, cache=None):
    """One call checked against the definition; returns (out, lse)."""
    import sliding_window_speculative_gb300 as swa
    scale = D ** -0.5 if scale is None else scale
    if cache is None:
        cache = Cache(B, Hkv, L, D, page, seed, spread)
    if poison:
        seen = np.zeros((B, L), bool)
        for b in range(B):
            lo, hi = max(0, q_pos[b] - W + 1), min(lens[b], L, q_pos[b] + q_len)
            seen[b, lo:max(hi, lo)] = True
        cache.poison(seen)
    cache.device()
    g = torch.Generator().manual_seed(seed + 100)
    q = (torch.randn((B, q_len, Hq, D), generator=g) * q_gain).to(torch.bfloat16)
    out, lse = swa.swa_q8_verify_attn(q.cuda(), *cache.dev, i32(lens), i32(q_pos), W, scale,
                                      block_table=cache.dev_table, num_splits=splits)
    torch.cuda.synchronize()
    assert swa.swa_read_device_errors() == 0
    k, v = cache.values(0), cache.values(1)
    for b in range(B):
        hi = min(lens[b], L, q_pos[b] + q_len)
        vis = np.s_[:, :max(hi, 0)]
        kb, vb = k[b][vis], v[b][vis]
        if hi <= 0:
            kb, vb = np.zeros((Hkv, 1, D)), np.zeros((Hkv, 1, D))
        o, z, mag, wv, seen = kv8.attention(q[b].double().numpy(), kb, vb, max(lens[b], 0), q_pos[b],
                                            W, scale)
        d = (D + 16) * 2.0 ** -24 * mag + 2.0 ** -20
        got_o, got_z = out[b].double().cpu().numpy(), lse[b].double().cpu().numpy()
        empty = np.isinf(z)
        assert np.array_equal(got_z == -np.inf, empty), b
        assert not np.abs(got_o[empty]).any(), b
        lo = max(0, q_pos[b] - W + 1)
        vmax = np.abs(vb[:, lo:]).max() if vb[:, lo:].size else 0.0
        tol = (2.0 ** -8 * np.abs(o) + (2 * d + 2.0 ** -8)[..., None] * wv +
               (seen * 2.0 ** -20)[..., None] * vmax)
        err = np.abs(got_o - o)
        assert np.all(err <= tol), (b, float((err / np.maximum(tol, 1e-300)).max()))
        ez = np.abs(got_z - z)[~empty]
        zt = (d + 2.0 ** -20 + 2.0 ** -22 * np.abs(z))[~empty]
        assert np.all(ez <= zt), (b, float((ez / zt).max()))
    return out, lse


KERNELS = ["plan", "simt", "tc", "rows"]
SHAPES = {
    # B, q_len, Hq, Hkv, D, W, L, lens, q_pos, page
    "one_key": (2, 1, 4, 2, 128, 1, 8, [1, 8], [0, 7], 0),
    "two_tokens": (1, 1, 8, 2, 256, 188, 64, [2], [1], 0),
    "verify_block": (2, 8, 8, 2, 256, 188, 512, [512, 400], [504, 392], 0),
    "tile_edges": (5, 2, 2, 1, 128, 127, 384, [130, 129, 128, 257, 384], [128, 127, 126, 255, 382], 0),
    "window_past_the_start": (2, 5, 6, 2, 256, 5000, 300, [300, 17], [295, 12], 0),
    "odd_paged": (3, 3, 9, 3, 128, 77, 240, [100, 233, 3], [97, 230, 0], 24),
    "pages_of_8": (2, 8, 8, 2, 256, 150, 256, [163, 256], [155, 248], 8),
    "empty_slots": (4, 4, 4, 4, 128, 64, 96, [0, 50, 0, 96], [0, 46, 0, 92], 0),
    "rows_past_the_end": (3, 6, 4, 2, 256, 16, 64, [10, 64, 5], [8, 62, 30], 16),
    "group_of_one": (2, 9, 3, 3, 128, 200, 320, [320, 210], [311, 201], 64),
    "group_of_eight": (2, 8, 16, 2, 256, 300, 512, [512, 301], [504, 293], 0),
    "long_block": (1, 64, 8, 2, 256, 188, 512, [500], [436], 16),
    "small_heads": (3, 4, 8, 4, 64, 333, 400, [400, 37, 1], [396, 33, 0], 8),
    "small_heads_block": (1, 64, 8, 2, 64, 100, 256, [256], [192], 0),
    "prefill": (1, 200, 4, 2, 128, 130, 512, [512], [312], 64),
    # more items than SMs, many of them per window: the plan reads bf16 rows
    "prefill_batch": (6, 130, 8, 2, 128, 100, 256, [256, 200, 130, 0, 7, 256],
                      [126, 70, 0, 0, 3, 120], 16),
    "prefill_batch_of_256": (3, 257, 8, 2, 256, 70, 320, [320, 257, 300], [63, 0, 40], 0),
    "prefill_batch_of_64": (6, 130, 8, 2, 64, 100, 256, [256, 200, 130, 0, 7, 256],
                            [126, 70, 0, 0, 3, 120], 0),
}


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("shape", list(SHAPES))
def test_attention_shapes(shape, kernel):
    B, q_len, Hq, Hkv, D, W, L, lens, q_pos, page = SHAPES[shape]
    with forced_kernel(kernel):
        _attend(B, q_len, Hq, Hkv, D, W, L, lens, q_pos, page)


@pytest.mark.parametrize("kernel", ["plan", "tc"])
@pytest.mark.parametrize("splits", [1, 2, 7, 64])
@pytest.mark.parametrize("page", [0, 16])
def test_attention_split_keys(splits, page, kernel):
    """The keys in chunks, some of them empty, merged by their sums."""
    with forced_kernel(kernel):
        _attend(3, 3, 8, 2, 128, 700, 1024, [1024, 600, 20], [1021, 597, 17], page, splits=splits)
        _attend(2, 2, 4, 2, 256, 400, 512, [512, 90], [510, 88], page, splits=splits)


@pytest.mark.parametrize("kernel", ["plan", "tc", "simt"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_attention_exponents_far_apart(D, kernel):
    """Keys and values of very different scales side by side, large scores,
    a zero and a negative scale."""
    with forced_kernel(kernel):
        _attend(2, 4, 4, 2, D, 150, 256, [256, 140], [252, 136], spread=20, seed=3, scale=1e-4)
        _attend(2, 4, 4, 2, D, 150, 256, [256, 140], [252, 136], seed=4, q_gain=30.0)
        _attend(1, 2, 4, 2, D, 150, 256, [256], [254], seed=5, scale=0.0)
        _attend(1, 2, 4, 2, D, 150, 256, [256], [254], seed=6, scale=-0.05)


@pytest.mark.parametrize("kernel", ["plan", "tc", "simt"])
def test_attention_of_queries_of_every_size(kernel):
    """Rows whose elements span what two e4m3 numbers hold, tiny and huge rows,
    zero rows: each row has a scale of its own."""
    import sliding_window_speculative_gb300 as swa
    B, q_len, Hq, Hkv, D, L = 1, 8, 4, 2, 256, 160
    cache = Cache(B, Hkv, L, D, seed=9)
    cache.device()
    rng = np.random.default_rng(7)
    q = rng.standard_normal((B, q_len, Hq, D))
    q[0, 0] *= 2.0 ** rng.integers(-20, 1, (Hq, D))
    q[0, 1] *= 1e-20
    q[0, 2] = 0
    q[0, 3, :, 1:] = 0
    q[0, 4] *= 2.0 ** -rng.integers(0, 10, (Hq, D))
    q[0, 5] *= 1e-39
    q = torch.from_numpy(q).to(torch.bfloat16)
    with forced_kernel(kernel):
        out, lse = swa.swa_q8_verify_attn(q.cuda(), *cache.dev, i32([L]), i32([L - 8]), 188, 0.0625)
    torch.cuda.synchronize()
    o, z, mag, wv, seen = kv8.attention(q[0].double().numpy(), cache.values(0)[0],
                                        cache.values(1)[0], L, L - 8, 188, 0.0625)
    d = (D + 16) * 2.0 ** -24 * mag + 2.0 ** -20
    assert np.all(np.abs(lse[0].double().cpu().numpy() - z) <= d + 2.0 ** -20 + 2.0 ** -22 * np.abs(z))
    tol = (2.0 ** -8 * np.abs(o) + (2 * d + 2.0 ** -8)[..., None] * wv +
           (seen * 2.0 ** -20)[..., None] * np.abs(cache.values(1)).max())
    assert np.all(np.abs(out[0].double().cpu().numpy() - o) <= tol)


@pytest.mark.parametrize("kernel", ["plan", "tc"])
def test_attention_of_one_heavy_key_without_values(kernel):
    """A first key that takes nearly all the weight and whose values are zero
    (or tiny): the others' weights, far smaller, still carry the result."""
    import sliding_window_speculative_gb300 as swa
    for tiny in (True, False):
        B, q_len, Hq, Hkv, D, L = 1, 2, 4, 2, 128, 300
        cache = Cache(B, Hkv, L, D, seed=11)
        cache.codes[1][:, :, 0] = 0 if tiny else 0x38
        cache.exps[1][:, :, 0] = -50 if tiny else -20
        cache.codes[0][:, :, 0] = 0x38                      # ones, times 2^e
        cache.exps[0][:, :, 0] = 0
        cache.device()
        q = torch.full((B, q_len, Hq, D), 0.125).to(torch.bfloat16)
        q += (torch.randn(q.shape, generator=torch.Generator().manual_seed(1)) * 0.01).to(q.dtype)
        with forced_kernel(kernel):
            out, lse = swa.swa_q8_verify_attn(q.cuda(), *cache.dev, i32([L]), i32([L - 2]), 400, 1.0)
        torch.cuda.synchronize()
        o, z, mag, wv, seen = kv8.attention(q[0].double().numpy(), cache.values(0)[0],
                                            cache.values(1)[0], L, L - 2, 400, 1.0)
        d = (D + 16) * 2.0 ** -24 * mag + 2.0 ** -20
        # (the small weights' floor, 2^-21 per key, counts from the largest
        # weight times its row's scale, not from the heavy key's weight)
        k, v = cache.values(0)[0], cache.values(1)[0]
        for i in range(q_len):
            for h in range(Hq):
                g = h // 2
                s = k[g, :L - 1 + i] @ q[0, i, h].double().numpy()
                w = np.exp(s - z[i, h])
                top = (w * 448 * 2.0 ** cache.exps[1][0, g, :L - 1 + i].astype(float)).max()
                tol = 2.0 ** -8 * np.abs(o[i, h]) + (2 * d[i, h] + 2.0 ** -8) * wv[i, h] + \
                    seen[i, h] * 2.0 ** -21 * top
                err = np.abs(out[0, i, h].double().cpu().numpy() - o[i, h])
                assert np.all(err <= tol), (tiny, i, h, float((err / tol).max()))


def test_attention_without_lse_and_into_given_outputs():
    import sliding_window_speculative_gb300 as swa
    cache = Cache(2, 2, 64, 128)
    cache.device()
    q = torch.randn((2, 4, 4, 128), device="cuda", dtype=torch.bfloat16)
    a, l = swa.swa_q8_verify_attn(q, *cache.dev, i32([64, 30]), i32([60, 26]), 40, 0.1)
    out = torch.full_like(q, 7.0)
    b, n = swa.swa_q8_verify_attn(q, *cache.dev, i32([64, 30]), i32([60, 26]), 40, 0.1, out=out,
                                  want_lse=False)
    assert n is None and b is out and torch.equal(a, b)


def test_equals_attention_over_the_rows_read_back():
    """The bf16 call on what swa_q8_read returns: the same definition on the
    same numbers."""
    import sliding_window_speculative_gb300 as swa
    B, L, W, q_len = 3, 256, 100, 8
    cache = Cache(B, 2, L, 256, 16, seed=21)
    cache.device()
    lens, pos = [256, 99, 150], [248, 91, 142]
    q = torch.randn((B, q_len, 8, 256), device="cuda", dtype=torch.bfloat16)
    out, lse = swa.swa_q8_verify_attn(q, *cache.dev, i32(lens), i32(pos), W, 0.0625,
                                      block_table=cache.dev_table)
    k, v = swa.swa_q8_read(*cache.dev, i32(lens), i32([0] * B), L, block_table=cache.dev_table)
    out2, lse2 = swa.swa_verify_attn(q, k, v, i32(lens), i32(pos), W, 0.0625)
    assert (lse - lse2).abs().max() < 1e-4
    assert (out.float() - out2.float()).abs().max() < 2.0 ** -6 * out2.float().abs().max()


def test_refusals_of_the_binding():
    import sliding_window_speculative_gb300 as swa
    cache = Cache(2, 2, 64, 128)
    k8, v8, ke, ve = cache.device()
    q = torch.zeros((2, 4, 4, 128), device="cuda", dtype=torch.bfloat16)
    kn = torch.zeros((2, 4, 2, 128), device="cuda", dtype=torch.bfloat16)
    lens, pos = i32([64, 30]), i32([60, 26])
    bad = [
        lambda: swa.swa_q8_verify_attn(q, k8.view(torch.uint8), v8, ke, ve, lens, pos, 8, 0.1),
        lambda: swa.swa_q8_verify_attn(q, k8, v8, ke.view(torch.uint8), ve, lens, pos, 8, 0.1),
        lambda: swa.swa_q8_verify_attn(q, k8, v8, ke[:, :, :32], ve, lens, pos, 8, 0.1),
        lambda: swa.swa_q8_verify_attn(q, k8, v8[:1], ke, ve, lens, pos, 8, 0.1),
        lambda: swa.swa_q8_verify_attn(q[..., :64].contiguous(), k8, v8, ke, ve, lens, pos, 8, 0.1),
        lambda: swa.swa_q8_verify_attn(q, k8, v8, ke, ve, lens[:1], pos, 8, 0.1),
        lambda: swa.swa_q8_verify_attn(q, k8, v8, ke, ve, lens.long(), pos, 8, 0.1),
        lambda: swa.swa_q8_verify_attn(q.float(), k8, v8, ke, ve, lens, pos, 8, 0.1),
        lambda: swa.swa_q8_append(kn[:, :, :1], kn[:, :, :1], k8, v8, ke, ve, lens, pos),
        lambda: swa.swa_q8_append(kn, kn[:1], k8, v8, ke, ve, lens, pos),
        lambda: swa.swa_q8_append(kn.transpose(1, 2), kn, k8, v8, ke, ve, lens, pos),
        lambda: swa.swa_q8_append(kn, kn, k8, v8, ke, ve, lens, pos[:1]),
        lambda: swa.swa_q8_read(k8, v8, ke, ve, lens, pos, 0),
        lambda: swa.swa_q8_read(k8, v8, ke, ve, lens, pos[:1], 4),
        lambda: swa.swa_q8_read(k8, v8, ke, ve, lens, pos, 4, k_out=kn),
        lambda: swa.swa_q8_verify_attn(q, k8, v8, ke, ve, lens, pos, 0, 0.1),
        lambda: swa.swa_q8_verify_attn(q, k8, v8, ke, ve, lens, pos, 8, float("nan")),
        lambda: swa.swa_q8_verify_attn(q, k8, v8, ke, ve, lens, pos, 8, 0.1,
                                       block_table=torch.zeros((2, 2), device="cuda")),
    ]
    for n, f in enumerate(bad):
        with pytest.raises((TypeError, ValueError, swa.SwaError)):
            f()
            pytest.fail(f"call {n} was taken")
