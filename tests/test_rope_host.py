"""Head norm + rotation without a GPU: argument refusals of the C entry
points (before any CUDA call) and of the binding, and the fp64 definition's
own invariants."""
import ctypes

import numpy as np
import pytest
import torch

import oracle.verify_step as vs
import sliding_window_speculative_gb300 as swa
from sliding_window_speculative_gb300 import build


@pytest.fixture(scope="module")
def lib():
    build.build()
    return swa.load_library()


GOOD_DIMS = (2, 8, 8, 2, 256, 4096, 0)
GOOD_ROPE = dict(q_row=13 * 256, k_row=13 * 256, v_row=13 * 256, q_weight=1024, k_weight=2048,
                 inv_freq=4096, eps=1e-6, rot_dim=256, interleaved=0)
PTRS = dict(q=16, k=32, v=48, q_pos=64, q_out=80, k_out=96, v_out=112)


def _rows(lib, dims=GOOD_DIMS, rope=(), **ptrs):
    r = None if rope is None else swa.SwaRope(**{**GOOD_ROPE, **dict(rope)})
    p = {**PTRS, **ptrs}
    d = None if dims is None else swa.make_dims(*dims)
    return lib.swa_qk_norm_rope(p["q"], p["k"], p["v"], None if r is None else ctypes.byref(r),
                                p["q_pos"], p["q_out"], p["k_out"], p["v_out"],
                                None if d is None else ctypes.byref(d), None)


def _append(lib, dims=GOOD_DIMS, rope=(), paged=None, **ptrs):
    r = swa.SwaRope(**{**GOOD_ROPE, **dict(rope)})
    p = {**PTRS, "k_cache": 128, "v_cache": 144, "seq_lens": 160, **ptrs}
    d = swa.make_dims(*dims)
    return lib.swa_qk_norm_rope_append(p["q"], p["k"], p["v"], ctypes.byref(r), p["k_cache"],
                                       p["v_cache"], None if paged is None else ctypes.byref(paged),
                                       p["seq_lens"], p["q_pos"], p["q_out"], ctypes.byref(d), None)


@pytest.mark.parametrize("call", [_rows, _append])
@pytest.mark.parametrize("dims,code", [
    ((0, 8, 8, 2, 256, 4096, 0), swa.SWA_ERR_INVALID_ARG),
    ((65536, 8, 8, 2, 256, 4096, 0), swa.SWA_ERR_INVALID_ARG),
    ((2, 0, 8, 2, 256, 4096, 0), swa.SWA_ERR_INVALID_ARG),
    ((2, 513, 8, 2, 256, 4096, 0), swa.SWA_ERR_INVALID_ARG),
    ((2, 8, 8, 3, 256, 4096, 0), swa.SWA_ERR_INVALID_ARG),
    ((2, 8, 8, 0, 256, 4096, 0), swa.SWA_ERR_INVALID_ARG),
    ((2, 8, 8, 2, 96, 4096, 0), swa.SWA_ERR_UNSUPPORTED),
])
def test_bad_dims(lib, call, dims, code):
    assert call(lib, dims) == code and swa.swa_last_error()


@pytest.mark.parametrize("call", [_rows, _append])
@pytest.mark.parametrize("rope", [
    {"rot_dim": 24}, {"rot_dim": 272}, {"rot_dim": -16}, {"interleaved": 2}, {"inv_freq": None},
    {"eps": 0.0}, {"eps": float("nan")}, {"eps": float("inf")}, {"q_row": 8 * 256 - 8},
    {"k_row": 13 * 256 + 4}, {"v_row": 0}, {"q_weight": 1028}, {"inv_freq": 4098},
])
def test_bad_rope(lib, call, rope):
    assert call(lib, rope=rope) == swa.SWA_ERR_INVALID_ARG and swa.swa_last_error()


@pytest.mark.parametrize("ptrs", [{n: None} for n in PTRS] + [{n: PTRS[n] + 2} for n in PTRS])
def test_bad_pointers(lib, ptrs):
    assert _rows(lib, **ptrs) == swa.SWA_ERR_INVALID_ARG
    assert _rows(lib, rope=None) == swa.SWA_ERR_INVALID_ARG
    assert _rows(lib, dims=None) == swa.SWA_ERR_INVALID_ARG


def test_append_refusals(lib):
    for name in ("k_cache", "v_cache", "seq_lens"):
        assert _append(lib, **{name: None}) == swa.SWA_ERR_INVALID_ARG
        assert _append(lib, **{name: 130}) == swa.SWA_ERR_INVALID_ARG
    assert _append(lib, dims=(2, 8, 8, 2, 256, 0, 0)) == swa.SWA_ERR_INVALID_ARG
    bad = [swa.SwaPaged(None, 256, 16, 600), swa.SwaPaged(64, 256, 12, 600),
           swa.SwaPaged(64, 255, 16, 600), swa.SwaPaged(64, 256, 16, 0), swa.SwaPaged(66, 256, 16, 9)]
    for p in bad:
        assert _append(lib, paged=p) == swa.SWA_ERR_INVALID_ARG


def test_binding_refuses_cpu_tensors():
    x = torch.zeros(1, 2, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA device"):
        swa.swa_qk_norm_rope(x, x, x, None, None, 1e-6, None, torch.zeros(1, dtype=torch.int32))


def test_definition_keeps_lengths_and_relative_angles():
    """Rotation keeps every pair's length, and the product of a rotated query
    and key depends on the distance of their positions alone."""
    rng = np.random.default_rng(0)
    x = rng.standard_normal((2, 1, 64))
    f = 10000.0 ** (-np.arange(16) / 16)
    for inter in (False, True):
        def dot(p, q):
            y, _ = vs.norm_rope(x, None, 0, f, [p, q], inter)
            assert np.allclose((y ** 2).sum(-1), (x ** 2).sum(-1))
            return float((y[0] * y[1]).sum())
        assert abs(dot(7, 3) - dot(1007, 1003)) < 1e-11
    y, _ = vs.norm_rope(x, np.ones(64), 0, None, [0, 1])
    assert np.allclose((y ** 2).mean(-1), 1)
