"""Attention over long windows of the 8-bit cache as the plan splits them, within bounds
that a result of zeros does not pass; pages of a tile and more; exactly the workspace that
swa_q8_workspace_bytes gives.

Bounds: see tests/test_q8_weights_gpu.py (each chunk's small weights are measured by its
own largest, so that the sum over chunks is within 7 sqrt(n) 2^-22 of the row's largest
for all n keys).  The bf16 rows that some blocks are attended over have weights within
2^-16: the same bounds hold."""
import numpy as np
import pytest
import torch

from tests.helpers import forced_kernel
from tests.q8_bounds import attention
from tests.test_q8_weights_gpu import bounds, codes_of, device_cache, i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import sliding_window_speculative_gb300 as swa
    from sliding_window_speculative_gb300 import build
    build.build()
    yield
    swa.swa_set_workspace(None)
    swa.swa_release_workspace()


class Case:
    """Normal keys, values with a common part (so that results of long windows stay well
    above their bounds), exponents that vary, nothing but NaN where no row looks."""

    def __init__(self, B, q_len, Hq, Hkv, D, W, L, page, lens=None, seed=0):
        rng = np.random.default_rng(seed + L + W)
        self.W, self.scale, self.page = W, D ** -0.5, page
        k = rng.standard_normal((B, Hkv, L, D), dtype=np.float32) * 110
        v = rng.standard_normal((B, Hkv, L, D), dtype=np.float32) * 50 + \
            rng.choice([-60.0, 60.0], (B, Hkv, 1, D))
        self.k8, self.v8 = codes_of(k.clip(-448, 448)), codes_of(v.clip(-448, 448))
        self.ke = rng.integers(-8, -5, (B, Hkv, L))
        self.ve = rng.integers(-8, -5, (B, Hkv, L))
        self.lens = lens or [L - 777 * b for b in range(B)]
        self.pos = [n - q_len for n in self.lens]
        for b in range(B):
            for x in (self.k8, self.v8):
                x[b, :, self.lens[b]:] = 0x7f
                x[b, :, :max(self.pos[b] - W + 1, 0)] = 0x7f
        q = rng.standard_normal((B, q_len, Hq, D))
        self.q = torch.from_numpy(q).to(torch.bfloat16)
        self.dev, self.table = device_cache(self.k8, self.v8, self.ke, self.ve, page, seed)

    def run(self, splits=0):
        import sliding_window_speculative_gb300 as swa
        out, lse = swa.swa_q8_verify_attn(self.q.cuda(), *self.dev, i32(self.lens), i32(self.pos),
                                          self.W, self.scale, block_table=self.table,
                                          num_splits=splits)
        torch.cuda.synchronize()
        assert swa.swa_read_device_errors() == 0
        return out, lse

    def check(self, got):
        if not hasattr(self, "want"):
            self.want = [attention(self.q[b].double().numpy(), self.k8[b], self.v8[b], self.ke[b],
                                   self.ve[b], self.lens[b], self.pos[b], self.W, self.scale)
                         for b in range(len(self.lens))]
        out, lse = (t.double().cpu().numpy() for t in got)
        for b, (o, z, mag, wv, top, seen) in enumerate(self.want):
            tol, zt = bounds(o, z, mag, wv, top, seen, self.q.shape[-1])
            tol += (7 * np.sqrt(seen) * 2.0 ** -22 * top)[..., None]
            err = np.abs(out[b] - o)
            assert np.all(err <= tol), (b, float((err / tol).max()))
            assert np.all(np.abs(lse[b] - z) <= zt), (b, float((np.abs(lse[b] - z) / zt).max()))
            assert (np.abs(o) > tol).mean() > 0.95


LONG = [
    # B, q_len, Hq, Hkv, D, W, L, page
    (1, 8, 8, 2, 256, 4096, 5120, 128),
    (2, 1, 16, 4, 128, 32768, 32768, 256),
    (1, 40, 8, 2, 128, 6000, 8192, 0),
    (3, 2, 8, 4, 64, 12031, 16384, 128),
    (1, 5, 9, 3, 256, 20000, 20480, 16),
    (1, 3, 4, 1, 128, 9000, 9216, 384),
]


@pytest.mark.parametrize("case", range(len(LONG)))
def test_windows_split_by_the_plan(case):
    """The plan splits these (a workspace that holds nothing is refused), and so does
    num_splits = 1 where the window is longer than a chunk may be."""
    import sliding_window_speculative_gb300 as swa
    c = Case(*LONG[case])
    W = LONG[case][5]
    try:
        swa.swa_set_workspace(torch.empty(16, dtype=torch.uint8, device="cuda"))
        with pytest.raises(swa.SwaError) as e:
            c.run()
        assert e.value.status == swa.SWA_ERR_WORKSPACE
        if W > 8192:
            with pytest.raises(swa.SwaError):
                c.run(1)
    finally:
        swa.swa_set_workspace(None)
    for kernel in ("plan", "tc"):
        with forced_kernel(kernel):
            for splits in (0, 1, 5):
                c.check(c.run(splits))


@pytest.mark.parametrize("page", [128, 136, 256, 1024])
@pytest.mark.parametrize("D,q_len,W", [(256, 8, 188), (128, 1, 600), (64, 3, 1000), (128, 200, 300)])
def test_pages_of_a_tile_and_more(D, q_len, W, page):
    L = page * (-(-1500 // page))
    c = Case(3, q_len, 8, 2, D, W, L, page, lens=[L, L - 129, max(q_len, 131)], seed=page)
    for kernel in ("plan", "tc", "rows"):
        with forced_kernel(kernel):
            c.check(c.run())


@pytest.mark.parametrize("args,splits,rows", [
    ((16, 64, 8, 2, 128, 188, 512, 0), 0, True),          # bf16 rows
    ((12, 64, 8, 2, 256, 100, 512, 16), 0, True),
    ((16, 64, 8, 2, 128, 188, 512, 0), 3, True),          # bf16 rows and partials
    ((2, 8, 8, 2, 256, 400, 512, 0), 5, False),           # partials
    ((1, 4, 8, 2, 64, 9000, 16384, 128), 1, False),       # more of them than asked for
])
def test_exactly_the_workspace_of_the_bound(args, splits, rows):
    """The bound's bytes are enough (and, of rows, needed); what lies behind them stays."""
    import sliding_window_speculative_gb300 as swa
    lens = [args[6] - 3 * b for b in range(args[0])]
    c = Case(*args, lens=lens)
    B, q_len, Hq, Hkv, D, W, L, page = args
    with forced_kernel("rows" if rows else "tc"):
        want = [t.clone() for t in c.run(splits)]
        c.check(want)
        need = swa.swa_q8_workspace_bytes(swa.make_dims(B, q_len, Hq, Hkv, D, L, splits), W)
        if rows:
            assert need >= 2 * B * Hkv * min(W + q_len - 1, L) * D * 2
        buf = torch.full((need + 4096,), 0x5a, dtype=torch.uint8, device="cuda")
        try:
            swa.swa_set_workspace(buf[:need])
            got = c.run(splits)
            assert (buf[need:] == 0x5a).all() and not (buf[:need] == 0x5a).all()
            assert all(torch.equal(a, b) for a, b in zip(got, want))
            if rows:
                swa.swa_set_workspace(buf[:2 * B * Hkv * min(W + q_len - 1, L) * D * 2])
                with pytest.raises(swa.SwaError) as e:
                    c.run(splits)
                assert e.value.status == swa.SWA_ERR_WORKSPACE
        finally:
            swa.swa_set_workspace(None)
