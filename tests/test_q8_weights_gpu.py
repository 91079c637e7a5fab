"""Weights of the attention straight from the 8-bit cache: their precision beside one
another and far below the largest one, over any number of keys.

Bounds, u = 2^-24, w_j the row's weights, e_j the exponent of V's row j:
  a score      d = (D + 16) u scale sum |q||k| + 2^-20 (products summed in fp32, three
               rounded factors, the exponential); the query rows here are e4m3 numbers
               or have no element below 2^-14 of their largest: exact
  a weight     e^d off, then held within 2^-14 of itself, or w_j 2^e_j within a step of
               2^-21 of its chunk's largest where that is more; a chunk has at most 8192
               keys.  The errors of that second kind are independent in effect (each
               key's rounding has an offset of its own, evenly spread over a step) and
               at most a step wide: n of them stay within 7 sqrt(n) half steps but for a
               chance of 2 e^-24 (Hoeffding), that is 7 sqrt(n) 2^-22 max_j(w_j 448 2^e_j)
  the sums     2^-21 of the summed magnitudes per MMA, 2^-22 more per 32 keys added on
  the result   2^-8 of itself (bf16), and two chunks or more joined in fp32: 2^-20
  lse          d + 2^-20 + n / 128 u (the row sum), 2^-22 of itself"""
import numpy as np
import pytest
import torch

from tests.helpers import forced_kernel
from tests.q8_bounds import attention

pytestmark = pytest.mark.gpu

E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sliding_window_speculative_gb300 import build
    build.build()
    yield


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def codes_of(x):
    """e4m3 codes of values that are within the format's range."""
    return torch.from_numpy(np.asarray(x)).float().to(E4M3).view(torch.uint8).numpy()


def device_cache(k8, v8, ke, ve, page, seed):
    """The cache on the device: ([k, v, k_exp, v_exp], table)."""
    B, Hkv, L, D = k8.shape
    arrays = [k8, v8, ke.astype(np.int8), ve.astype(np.int8)]
    if not page:
        dev, table = [torch.from_numpy(a).cuda() for a in arrays], None
    else:
        nb = L // page
        table = np.random.default_rng(seed).permutation(B * nb).astype(np.int32)
        dev = []
        for a in arrays:
            pool = np.empty((B * nb, Hkv, page) + a.shape[3:], a.dtype)
            pool[table] = np.moveaxis(a.reshape((B, Hkv, nb, page) + a.shape[3:]), 1, 2).reshape(
                pool.shape)
            dev.append(torch.from_numpy(pool).cuda())
        table = torch.from_numpy(table.reshape(B, nb)).cuda()
    return [dev[0].view(E4M3), dev[1].view(E4M3), dev[2], dev[3]], table


def bounds(o, z, mag, wv, top, seen, D):
    """Tolerances of out and lse of rows whose small weights are one chunk's."""
    d = (D + 16) * 2.0 ** -24 * mag + 2.0 ** -20
    n = np.minimum(seen, 8192)
    tol = ((2.0 ** -8 + 2.0 ** -20) * np.abs(o) + (7 * np.sqrt(n) * 2.0 ** -22 * top)[..., None] +
           (2 * d + 2.0 ** -14 + 2.0 ** -21 + n / 32 * 2.0 ** -22)[..., None] * wv)
    return tol, d + 2.0 ** -20 + n / 128 * 2.0 ** -24 + 2.0 ** -22 * np.abs(z)


def run(q, cache, table, lens, pos, W, scale, splits=0):
    import sliding_window_speculative_gb300 as swa
    out, lse = swa.swa_q8_verify_attn(q.cuda(), *cache, i32(lens), i32(pos), W, scale,
                                      block_table=table, num_splits=splits)
    torch.cuda.synchronize()
    assert swa.swa_read_device_errors() == 0
    return out.double().cpu().numpy(), lse.double().cpu().numpy()


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("n", [2, 3, 9])
def test_weights_that_cancel(D, n):
    """Few keys of nearly equal weights whose V elements are + or - one size: where they
    cancel the weights' own rounding is all that is left (at 11 bits it would be four
    times the bound)."""
    B, q_len, Hq, Hkv = 16, 8, 8, 2
    rng = np.random.default_rng(D + n)
    k8 = codes_of(rng.standard_normal((B, Hkv, n, D)) * 20)
    v8 = codes_of(rng.choice([-256.0, 256.0], (B, Hkv, n, D)))
    ke = np.full((B, Hkv, n), -8)
    ve = np.full((B, Hkv, n), -8)
    q = torch.from_numpy(rng.integers(-7, 8, (B, q_len, Hq, D)) * 2.0 ** -3).to(torch.bfloat16)
    cache, table = device_cache(k8, v8, ke, ve, 0, 0)
    lens, pos = [n] * B, [n - 1] * B            # (later rows see the same keys)
    scale = 0.05
    with forced_kernel("tc"):
        out, lse = run(q, cache, table, lens, pos, 64, scale)
    least = np.inf
    for b in range(B):
        o, z, mag, wv, top, seen = attention(q[b].double().numpy(), k8[b], v8[b], ke[b], ve[b], n,
                                             n - 1, 64, scale)
        tol, zt = bounds(o, z, mag, wv, top, seen, D)
        err = np.abs(out[b] - o)
        assert np.all(err <= tol), (b, float((err / tol).max()))
        assert np.all(np.abs(lse[b] - z) <= zt), b
        least = min(least, tol.min())
    # (the bound is one that 11 bits break; an odd number of + and - leaves 1 / n)
    assert n % 2 or least < 2.0 ** -12, least


@pytest.mark.parametrize("D,L,page", [(128, 32768, 0), (256, 32768, 16), (64, 40000, 0),
                                      (128, 131072, 128)])
@pytest.mark.parametrize("nats", [11.0, 13.0, 15.2, 16.5])
def test_one_heavy_key_and_a_long_tail(D, L, page, nats):
    """A key that takes nearly all the weight, all others alike and far below it: their
    sum is what half of the dims hold, V has one sign.  The bound does not grow with the
    number of keys."""
    B, q_len, Hq, Hkv, at = 1, 2, 4, 1, 1000
    rng = np.random.default_rng(L)
    qv = 0.5
    k = np.zeros((B, Hkv, L, D))
    k[..., :8] = 0.5 * rng.integers(0, 3, (B, Hkv, L, 8)) / 8     # scores of their own
    k[0, 0, at, :] = 0
    k[0, 0, at, 8:24] = 16.0
    v = rng.uniform(128, 256, (B, Hkv, L, D))
    v[0, 0, at, D // 2:] = 0
    k8, v8 = codes_of(k), codes_of(v)
    ke, ve = np.zeros((B, Hkv, L), int), np.full((B, Hkv, L), -8)
    q = torch.full((B, q_len, Hq, D), qv).to(torch.bfloat16)
    scale = nats / (16 * 16.0 * qv)
    cache, table = device_cache(k8, v8, ke, ve, page, 3)
    o, z, mag, wv, top, seen = attention(q[0].double().numpy(), k8[0], v8[0], ke[0], ve[0], L,
                                         L - q_len, L, scale)
    # (the others differ by a factor of 2 at most: in the chunks without the heavy key
    # all weights are far above a step of their largest)
    assert np.exp(8 * qv * 0.125 * scale) < 2
    tol, zt = bounds(o, z, mag, wv, top, seen, D)
    tail = np.abs(o[..., D // 2:])
    assert np.median(tol[..., D // 2:] / tail) < 0.25
    for kernel in ("plan", "tc"):
        for splits in (0, 1):
            with forced_kernel(kernel):
                out, lse = run(q, cache, table, [L], [L - q_len], L, scale, splits)
            err = np.abs(out[0] - o)
            assert np.all(err <= tol), (kernel, splits, float((err / tol).max()))
            assert np.all(np.abs(lse[0] - z) <= zt), (kernel, splits)
