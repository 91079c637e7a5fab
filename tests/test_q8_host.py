"""The 8-bit cache and the token log probabilities without a GPU: refusals of
the C entry points (before any CUDA call) and of the binding, the workspace
bound, and the fp64 definitions' own invariants."""
import ctypes

import numpy as np
import pytest
import torch

import oracle.kv8 as kv8
import sliding_window_speculative_gb300 as swa
from sliding_window_speculative_gb300 import build


@pytest.fixture(scope="module")
def lib():
    build.build()
    return swa.load_library()


DIMS = (2, 8, 8, 2, 256, 4096, 0)
CACHE = dict(k=16, v=32, k_exp=49, v_exp=51)
PTRS = dict(k_new=64, v_new=80, seq_lens=96, q_pos=112, start=128, k_out=144, v_out=160, q=176,
            out=192, lse=208)
ROW = 12 * 256


def _cache(over):
    return None if over is None else ctypes.byref(swa.SwaQ8Cache(**{**CACHE, **over}))


def _ref(x):
    return None if x is None else ctypes.byref(x)


def _append(lib, dims=DIMS, cache=(), paged=None, k_row=ROW, v_row=ROW, **ptrs):
    p = {**PTRS, **ptrs}
    return lib.swa_q8_append(p["k_new"], p["v_new"], k_row, v_row,
                             _cache(None if cache is None else dict(cache)), _ref(paged),
                             p["seq_lens"], p["q_pos"],
                             None if dims is None else ctypes.byref(swa.make_dims(*dims)), None)


def _read(lib, dims=DIMS, cache=(), paged=None, n=5, **ptrs):
    p = {**PTRS, **ptrs}
    return lib.swa_q8_read(_cache(None if cache is None else dict(cache)), _ref(paged),
                           p["seq_lens"], p["start"], n, p["k_out"], p["v_out"],
                           None if dims is None else ctypes.byref(swa.make_dims(*dims)), None)


def _verify(lib, dims=DIMS, cache=(), paged=None, window=188, scale=0.0625, **ptrs):
    p = {**PTRS, **ptrs}
    return lib.swa_q8_verify_attn(p["q"], _cache(None if cache is None else dict(cache)),
                                  _ref(paged), p["seq_lens"], p["q_pos"], window, scale, p["out"],
                                  p["lse"],
                                  None if dims is None else ctypes.byref(swa.make_dims(*dims)), None)


CALLS = [_append, _read, _verify]
INV, UNS = swa.SWA_ERR_INVALID_ARG, swa.SWA_ERR_UNSUPPORTED


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("dims,code", [
    (None, INV), ((0, 8, 8, 2, 256, 4096, 0), INV), ((65536, 8, 8, 2, 256, 4096, 0), INV),
    ((2, 8, 8, 0, 256, 4096, 0), INV), ((2, 8, 8, 2, 96, 4096, 0), UNS),
    ((2, 8, 8, 2, 256, 0, 0), INV), ((2, 8, 70000, 70000, 256, 64, 0), INV),
])
def test_bad_dims(lib, call, dims, code):
    assert call(lib, dims=dims) == code and swa.swa_last_error()


@pytest.mark.parametrize("call", [_append, _verify])
@pytest.mark.parametrize("q_len", [0, -1, 513])
def test_bad_block_length(lib, call, q_len):
    assert call(lib, dims=(2, q_len, 8, 2, 256, 4096, 0)) == INV


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("cache", [None, {"k": None}, {"v": None}, {"k_exp": None},
                                   {"v_exp": None}, {"k": 24}, {"v": 40}])
def test_bad_caches(lib, call, cache):
    assert call(lib, cache=cache) == INV and swa.swa_last_error()


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("paged", [
    swa.SwaPaged(None, 256, 16, 600), swa.SwaPaged(64, 256, 12, 600), swa.SwaPaged(64, 255, 16, 600),
    swa.SwaPaged(64, 256, 16, 0), swa.SwaPaged(66, 256, 16, 9)])
def test_bad_pages(lib, call, paged):
    assert call(lib, paged=paged) == INV


def test_huge_pools_refused(lib):
    pool = swa.SwaPaged(64, 256, 16, 1 << 27)
    for call in CALLS:
        assert call(lib, paged=pool) == UNS


@pytest.mark.parametrize("call,names", [
    (_append, ("k_new", "v_new", "seq_lens", "q_pos")),
    (_read, ("seq_lens", "start", "k_out", "v_out")),
    (_verify, ("q", "seq_lens", "q_pos", "out"))])
def test_bad_pointers(lib, call, names):
    for n in names:
        assert call(lib, **{n: None}) == INV, n
        assert call(lib, **{n: PTRS[n] + 2}) == INV, n


def test_other_refusals(lib):
    for row in (2 * 256 - 8, ROW + 4, 0, -ROW):
        assert _append(lib, k_row=row) == INV and _append(lib, v_row=row) == INV
    assert _read(lib, n=0) == INV and _read(lib, n=-3) == INV
    assert _verify(lib, window=0) == INV
    for s in (float("nan"), float("inf"), float("-inf")):
        assert _verify(lib, scale=s) == INV
    assert _verify(lib, lse=210) == INV
    assert _verify(lib, dims=(2, 8, 8, 3, 256, 4096, 0)) == INV
    assert _verify(lib, dims=(2, 64, 512, 1, 256, 4096, 0)) == UNS


def test_workspace_bound(lib):
    assert swa.swa_q8_workspace_bytes(swa.make_dims(*DIMS), 188) > 0
    assert swa.swa_q8_workspace_bytes(swa.make_dims(0, 8, 8, 2, 256, 4096), 188) == 0
    assert swa.swa_q8_workspace_bytes(swa.make_dims(*DIMS), 0) == 0
    # heads of 64, or one item of 32 packed rows per window: partials at most; otherwise
    # the windows' bf16 rows as well
    for D, q_len, rows in ((64, 512, False), (128, 8, False), (256, 8, False), (256, 16, False),
                           (128, 64, True), (256, 64, True), (128, 16, True)):
        dims = swa.make_dims(16, q_len, 8, 2, D, 4096)
        window = 188
        need, parts = swa.swa_q8_workspace_bytes(dims, window), swa.swa_workspace_bytes(dims, window)
        span = 2 * 16 * 2 * (window + q_len - 1) * D * 2
        assert need == parts if not rows else need >= span + parts, (D, q_len)
    # a long window at two items reads in place
    dims = swa.make_dims(16, 16, 8, 2, 128, 4096)
    assert swa.swa_q8_workspace_bytes(dims, 1024) == swa.swa_workspace_bytes(dims, 1024)


LOGP = dict(logits=2, keep_ids=None, tokens=16, temperature=None, logprobs=32, ranks=48, entropy=64,
            top_tokens=80, top_logprobs=96)


def _logprobs(lib, top=4, batch=2, q_len=8, vocab=1000, **ptrs):
    p = {**LOGP, **ptrs}
    return lib.swa_token_logprobs(p["logits"], p["keep_ids"], p["tokens"], p["temperature"], top,
                                  p["logprobs"], p["ranks"], p["entropy"], p["top_tokens"],
                                  p["top_logprobs"], batch, q_len, vocab, None)


@pytest.mark.parametrize("bad", [
    {"batch": 0}, {"batch": 65536}, {"q_len": 0}, {"q_len": 513}, {"vocab": 0}, {"vocab": -5},
    {"top": -1}, {"top": 33}, {"top": 8, "vocab": 7}, {"logits": None}, {"logits": 3},
    {"tokens": None}, {"tokens": 18}, {"logprobs": None}, {"logprobs": 34}, {"ranks": 50},
    {"entropy": 66}, {"top_tokens": None}, {"top_logprobs": None}, {"top_tokens": 82},
    {"keep_ids": 17}, {"temperature": 21}])
def test_logprobs_refusals(lib, bad):
    assert _logprobs(lib, **bad) == INV and swa.swa_last_error()


def test_binding_refuses_cpu_tensors():
    z = lambda *s, dt=torch.bfloat16: torch.zeros(s, dtype=dt)  # noqa: E731
    c = (z(1, 2, 16, 64).to(torch.float8_e4m3fn), z(1, 2, 16, 64).to(torch.float8_e4m3fn),
         z(1, 2, 16, dt=torch.int8), z(1, 2, 16, dt=torch.int8))
    one = z(1, dt=torch.int32)
    with pytest.raises(ValueError, match="CUDA device"):
        swa.swa_q8_append(z(1, 4, 2, 64), z(1, 4, 2, 64), *c, one, one)
    with pytest.raises(ValueError, match="CUDA device"):
        swa.swa_q8_read(*c, one, one, 4)
    with pytest.raises(ValueError, match="CUDA device"):
        swa.swa_q8_verify_attn(z(1, 4, 4, 64), *c, one, one, 8, 0.125)
    with pytest.raises(ValueError, match="CUDA device"):
        swa.swa_token_logprobs(z(1, 4, 100), z(1, 4, dt=torch.int32))


# ---------------------------------------------------------- the definitions

def test_e4m3_values_are_the_formats():
    codes = torch.arange(256, dtype=torch.uint8)
    want = codes.view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(kv8.E4M3, want, equal_nan=True)
    assert np.array_equal(np.signbit(kv8.E4M3), np.signbit(want)) or np.isnan(want[127])


def test_quantised_rows():
    rng = np.random.default_rng(3)
    for scale in (1e-30, 1e-12, 1.0, 37.0, 1e12):
        x = torch.from_numpy(rng.standard_normal(256) * scale).to(torch.bfloat16)
        code, e = kv8.quantise_row(x.double().numpy())
        back = kv8.row_values(code, np.array(e))
        a = np.abs(x.double().numpy()).max()
        assert a <= 448 * 2.0 ** e and (e == kv8.E_MIN or a > 448 * 2.0 ** (e - 1))
        # nearest: half a step of four significant bits, or of the smallest numbers
        err = np.abs(back - x.double().numpy())
        assert np.all(err <= np.maximum(2.0 ** -4 * np.abs(x.double().numpy()), 2.0 ** (e - 10)))
        # the values are bf16 numbers
        assert np.array_equal(torch.from_numpy(back).to(torch.bfloat16).double().numpy(), back)
        # torch's conversion of the scaled row
        t = (x.float() * 2.0 ** -e).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
        assert np.array_equal(t, code)
    code, e = kv8.quantise_row([0.0, np.inf, np.nan, -3.5, -np.inf])
    assert code.tolist() == [0, 127, 127, 0xfe, 127] and e == -7
    assert kv8.quantise_row([0.0, -0.0])[1] == -50
    assert kv8.quantise_row([1e30])[0][0] == 0x7e and kv8.quantise_row([1e30])[1] == 50


def test_logprob_row_against_log_softmax():
    rng = np.random.default_rng(4)
    x = rng.standard_normal(500) * 3
    x[[7, 9]] = 20.0
    for T in (1.0, 0.5, 0.0):
        lp, rank, ent, names, tops = kv8.logprob_row(x, 9, T, 3)
        p = torch.log_softmax(torch.from_numpy(x) / (T or 1.0), 0)
        assert abs(lp - p[9].item()) < 1e-12 and rank == 2 and names[:2].tolist() == [7, 9]
        assert abs(ent + (p.exp() * p).sum().item()) < 1e-12
        assert np.allclose(tops[:2], p[9].item())
    assert kv8.logprob_row(x, 500)[:2] == (-np.inf, 0)
    assert kv8.logprob_row(np.full(4, -np.inf), 2)[:3] == (-np.inf, 3, 0.0)
    lp, rank, ent, _, _ = kv8.logprob_row([1.0, np.inf, np.nan, np.inf], 3)
    assert rank == 2 and np.isclose(lp, -np.log(2)) and np.isclose(ent, np.log(2))
