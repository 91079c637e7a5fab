"""Attention rows whose scores rise from tile to tile, so that nearly every tile raises
the rows' reference maxima and the accumulators in tensor memory are scaled between two
MMAs into them: the key-major kernels over the bf16 and the 8-bit cache.

Bounds, u = 2^-24, w_j the row's weights: a score is off by d = (D + 16) u scale
sum |q||k| + 2^-20 (products summed in fp32, the exponential), a weight by e^d and its
rounding (11 bits or more: 2^-11, or 2^-21 of the largest w_j 448 2^e_j where that is
more), the accumulation by 2^-21 and 2^-22 per 32 keys, the result by 2^-8 (bf16); lse by
d + 2^-20 + 2^-22 of itself."""
import numpy as np
import pytest
import torch

import oracle.kv8 as kv8
from tests.helpers import forced_kernel
from tests.q8_bounds import attention

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sliding_window_speculative_gb300 import build
    build.build()
    yield


E4M3 = torch.float8_e4m3fn


def _rising(B, q_len, Hq, Hkv, D, L, shape, seed):
    """q, k, v whose scores (scale D^-0.5) climb about 10 log2 units per 128 keys."""
    rng = np.random.default_rng(seed)
    j = np.arange(L) / L
    a = {"rising": j, "zigzag": np.where(np.arange(L) // 128 % 2 == 0, j, j / 2),
         "falling": 1 - j}[shape]
    u = rng.choice([-1.0, 1.0], D)
    gain = 10 * (L / 128) / 1.4427 / D ** 0.5
    k = a[None, None, :, None] * u + rng.standard_normal((B, Hkv, L, D)) * 0.02
    q = gain * u * (1 + 0.05 * rng.standard_normal((B, q_len, Hq, 1))) + \
        rng.standard_normal((B, q_len, Hq, D)) * 0.1
    v = rng.standard_normal((B, Hkv, L, D))
    return [torch.from_numpy(x).to(torch.bfloat16) for x in (q, k, v)]


def _check(got, q, k8, v8, ke, ve, lens, pos, W):
    out, lse = (t.double().cpu().numpy() for t in got)
    D = q.shape[-1]
    for b in range(len(lens)):
        o, z, mag, wv, top, seen = attention(q[b].double().numpy(), k8[b], v8[b], ke[b], ve[b],
                                             lens[b], pos[b], W, D ** -0.5)
        d = (D + 16) * 2.0 ** -24 * mag + 2.0 ** -20
        tol = (2.0 ** -8 * np.abs(o) +
               (2 * d + 2.0 ** -11 + 2.0 ** -21 + seen / 32 * 2.0 ** -22)[..., None] * wv +
               (seen * 2.0 ** -21 * top)[..., None])
        err = np.abs(out[b] - o)
        assert np.all(err <= tol), (b, float((err / tol).max()))
        ez = np.abs(lse[b] - z)
        assert np.all(ez <= d + 2.0 ** -20 + 2.0 ** -22 * np.abs(z)), (b, float(ez.max()))
        # (a result without its last tiles would not pass)
        assert (np.abs(o) > tol).mean() > 0.9


@pytest.mark.parametrize("shape", ["rising", "zigzag", "falling"])
@pytest.mark.parametrize("B,q_len,Hq,Hkv,D,L,W,page", [
    (2, 8, 8, 2, 256, 1400, 1300, 0), (3, 1, 4, 2, 128, 1400, 5000, 16),
    (2, 4, 8, 2, 64, 1100, 1000, 0), (1, 24, 8, 2, 128, 1400, 1200, 8)])
def test_the_8_bit_cache(B, q_len, Hq, Hkv, D, L, W, page, shape):
    import sliding_window_speculative_gb300 as swa
    L = L // 16 * 16
    q, k, v = _rising(B, q_len, Hq, Hkv, D, L, shape, D + B)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    sh, table = ((B * L // page, Hkv, page), torch.randperm(B * L // page).view(B, -1).int().cuda()) \
        if page else ((B, Hkv, L), None)
    cache = [torch.zeros((*sh, D), dtype=torch.uint8, device="cuda").view(E4M3) for _ in range(2)]
    cache += [torch.zeros(sh, dtype=torch.int8, device="cuda") for _ in range(2)]
    for at in range(0, L, 512):                       # (an append takes up to 512 tokens)
        new = [x[:, :, at:at + 512].transpose(1, 2).contiguous().cuda() for x in (k, v)]
        n = new[0].shape[1]
        swa.swa_q8_append(*new, *cache, i32([at + n] * B), i32([at] * B), block_table=table)
    codes = [[kv8.quantise_row(x[b, h, j].double().numpy()) for b in range(B) for h in range(Hkv)
              for j in range(L)] for x in (k, v)]
    k8, v8 = (np.stack([c for c, _ in x]).reshape(B, Hkv, L, D) for x in codes)
    ke, ve = (np.array([e for _, e in x]).reshape(B, Hkv, L) for x in codes)
    lens = [L - 37 * b for b in range(B)]
    pos = [n - q_len for n in lens]
    for kernel in ("plan", "tc"):
        for splits in (1, 3):
            with forced_kernel(kernel):
                call = lambda: swa.swa_q8_verify_attn(  # noqa: E731
                    q.cuda(), *cache, i32(lens), i32(pos), W, D ** -0.5, block_table=table,
                    num_splits=splits)
                got, again = call(), call()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, again))
            _check(got, q, k8, v8, ke, ve, lens, pos, W)
    assert swa.swa_read_device_errors() == 0


@pytest.mark.parametrize("shape", ["rising", "zigzag", "falling"])
@pytest.mark.parametrize("B,q_len,Hq,Hkv,D,L,W", [
    (2, 8, 8, 2, 256, 1400, 1300), (3, 1, 4, 2, 128, 1400, 5000), (1, 24, 8, 2, 128, 1400, 1200)])
def test_the_bf16_cache(B, q_len, Hq, Hkv, D, L, W, shape):
    """The same of swa_verify_attn, on rows that are e4m3 numbers times 2^-6 already."""
    import sliding_window_speculative_gb300 as swa
    q, k, v = _rising(B, q_len, Hq, Hkv, D, L, shape, D + B)
    k8, v8 = ((x.float() * 64).clamp(-448, 448).to(E4M3) for x in (k, v))
    kd, vd = ((x.float() / 64).to(torch.bfloat16).cuda() for x in (k8, v8))
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    lens = [L - 37 * b for b in range(B)]
    pos = [n - q_len for n in lens]
    ex = np.full((B, Hkv, L), -6)
    codes = [x.view(torch.uint8).numpy() for x in (k8, v8)]
    for kernel in ("tc", "rows"):
        with forced_kernel(kernel):
            call = lambda: swa.swa_verify_attn(q.cuda(), kd, vd, i32(lens), i32(pos), W,  # noqa: E731
                                               D ** -0.5, num_splits=1)
            got, again = call(), call()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, again))
        _check(got, q, *codes, ex, ex, lens, pos, W)
    assert swa.swa_read_device_errors() == 0
