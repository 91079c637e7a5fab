"""Attention straight from the 8-bit cache with infinities, NaN and values at the ends of
the range in what it reads: rows that see them become NaN, all others keep their bits."""
import numpy as np
import pytest
import torch

from tests.helpers import forced_kernel

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


def inputs(B, q_len, Hq, Hkv, D, L, seed=0):
    """q on the host, the cache on the device (codes of normal values, exponents -9..-7)."""
    rng = np.random.default_rng(seed)
    q = torch.from_numpy(rng.standard_normal((B, q_len, Hq, D))).to(torch.bfloat16)
    cache = [torch.from_numpy(rng.standard_normal((B, Hkv, L, D)) * 110).float().clamp(-448, 448)
             .to(E4M3).view(torch.uint8).cuda() for _ in range(2)]
    cache += [torch.from_numpy(rng.integers(-9, -6, (B, Hkv, L)).astype(np.int8)).cuda()
              for _ in range(2)]
    return q, cache


def call(q, cache, lens, pos, W, scale, **kw):
    import sliding_window_speculative_gb300 as swa
    with forced_kernel("tc"):
        out, lse = swa.swa_q8_verify_attn(q.cuda(), cache[0].view(E4M3), cache[1].view(E4M3),
                                          cache[2], cache[3], i32(lens), i32(pos), W, scale, **kw)
    torch.cuda.synchronize()
    assert swa.swa_read_device_errors() == 0
    return out.cpu(), lse.cpu()


SHAPES = [(2, 8, 8, 2, 256, 300, 188), (2, 3, 4, 2, 128, 300, 400), (1, 24, 4, 4, 64, 200, 90)]


@pytest.mark.parametrize("value", [float("inf"), -float("inf"), float("nan")])
@pytest.mark.parametrize("splits", [1, 2])
@pytest.mark.parametrize("B,q_len,Hq,Hkv,D,L,W", SHAPES)
def test_infinities_and_nan_in_a_query_row(B, q_len, Hq, Hkv, D, L, W, splits, value):
    """0 times infinity is NaN, and so is a softmax of infinities."""
    q, cache = inputs(B, q_len, Hq, Hkv, D, L, seed=D)
    for t in cache[:2]:
        t[..., 5] = 0                             # (a dim that is zero in every key)
    lens, pos = [L - 13 * b for b in range(B)], [L - 13 * b - q_len for b in range(B)]
    want = call(q, cache, lens, pos, W, D ** -0.5, num_splits=splits)
    bad = torch.zeros((B, q_len, Hq), dtype=torch.bool)
    for b, i, h, d in ((0, 0, 0, 5), (0, q_len - 1, Hq - 1, 7), (B - 1, q_len // 2, 1, D - 1)):
        q[b, i, h, d] = value
        bad[b, i, h] = True
    out, lse = call(q, cache, lens, pos, W, D ** -0.5, num_splits=splits)
    assert out[bad].isnan().all() and lse[bad].isnan().all()
    assert torch.equal(out[~bad], want[0][~bad]) and torch.equal(lse[~bad], want[1][~bad])
    # a row that sees no key looks at nothing
    out, lse = call(q, cache, [0] * B, [0] * B, W, D ** -0.5, num_splits=splits)
    assert not out.any() and (lse == -float("inf")).all()


@pytest.mark.parametrize("m", [-100, -60, 60, 110, 119])
@pytest.mark.parametrize("B,q_len,Hq,Hkv,D,L,W", SHAPES)
def test_queries_of_every_magnitude(B, q_len, Hq, Hkv, D, L, W, m):
    """Queries times 2^m under a scale of 2^-m: no step between them may leave the range,
    and every product with a power of two is exact, so the bits are the same."""
    q, cache = inputs(B, q_len, Hq, Hkv, D, L, seed=D + 1)
    cache[2] += 10
    # (a whole number of steps, so that 2^m times it is a bf16 number, at most 8)
    q = (q.float() * 16).round().clamp(-128, 128) / 16
    lens, pos = [L] * B, [L - q_len] * B
    want = call(q.to(torch.bfloat16), cache, lens, pos, W, 2.0 ** -4)
    big = (q.double() * 2.0 ** m).to(torch.bfloat16)
    assert torch.equal(big.double(), q.double() * 2.0 ** m)
    got = call(big, cache, lens, pos, W, 2.0 ** (-4 - m))
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    assert want[0].isfinite().all() and want[1].isfinite().all()


@pytest.mark.parametrize("code", [0x7f, 0xff])
@pytest.mark.parametrize("kernel", ["tc", "rows"])
@pytest.mark.parametrize("B,q_len,Hq,Hkv,D,L,W", SHAPES)
def test_nan_in_a_visible_key(B, q_len, Hq, Hkv, D, L, W, code, kernel):
    """A NaN in K makes the rows NaN that see it, in V their dim; rows of the block that do
    not see it keep theirs (of V, the other dims: weights of 0 are multiplied too)."""
    import sliding_window_speculative_gb300 as swa
    if D == 64 and kernel == "rows":
        pytest.skip("heads of 64 have no such kernel")
    q, cache = inputs(B, q_len, Hq, Hkv, D, L, seed=D + 2)
    lens, pos = [L] * B, [L - q_len] * B
    G, last, d = Hq // Hkv, L - 1, 3                 # (only the block's last row sees L - 1)

    def run(cache):
        with forced_kernel(kernel):
            out, lse = swa.swa_q8_verify_attn(q.cuda(), cache[0].view(E4M3), cache[1].view(E4M3),
                                              cache[2], cache[3], i32(lens), i32(pos), W, D ** -0.5)
        torch.cuda.synchronize()
        assert swa.swa_read_device_errors() == 0
        return out.cpu(), lse.cpu()

    want = run(cache)
    bad = [t.clone() for t in cache]
    bad[0][0, 0, last, d] = code
    out, lse = run(bad)
    sees = torch.zeros((B, q_len, Hq), dtype=torch.bool)
    sees[0, q_len - 1, :G] = True
    assert out[sees].isnan().all()
    assert torch.equal(out[~sees], want[0][~sees]) and torch.equal(lse[~sees], want[1][~sees])
    bad = [t.clone() for t in cache]
    bad[1][0, 0, last, d] = code
    out, lse = run(bad)
    assert out[sees][:, d].isnan().all() and torch.equal(lse, want[1])
    same = torch.ones_like(out, dtype=torch.bool)
    same[0, :, :G, d] = False                        # (may be NaN in the block's other rows)
    assert torch.equal(out[same], want[0][same])
