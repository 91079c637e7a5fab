"""Sink attention without a GPU: refusals before any CUDA call, and the fp64
definition against the windowed oracle."""
import ctypes

import numpy as np
import pytest
import torch

import oracle
import oracle.verify_step as vs
import sliding_window_speculative_gb300 as swa
from sliding_window_speculative_gb300 import build


@pytest.fixture(scope="module")
def lib():
    build.build()
    return swa.load_library()


def _call(lib, dims=(2, 8, 8, 2, 256, 4096, 0), window=188, sinks=4, k_new=None, v_new=None,
          paged=None, scale=0.0625, q=16, k=32, v=48, sl=64, qp=80, out=96, lse=None):
    d = swa.make_dims(*dims)
    return lib.swa_sink_verify_attn(q, k_new, v_new, k, v,
                                    None if paged is None else ctypes.byref(paged), sl, qp, window,
                                    sinks, scale, out, lse, ctypes.byref(d), None)


@pytest.mark.parametrize("kw,code", [
    (dict(sinks=-1), swa.SWA_ERR_INVALID_ARG), (dict(sinks=129), swa.SWA_ERR_UNSUPPORTED),
    (dict(window=0), swa.SWA_ERR_INVALID_ARG), (dict(q=None), swa.SWA_ERR_INVALID_ARG),
    (dict(out=None), swa.SWA_ERR_INVALID_ARG), (dict(k=40), swa.SWA_ERR_INVALID_ARG),
    (dict(k_new=112), swa.SWA_ERR_INVALID_ARG), (dict(v_new=112), swa.SWA_ERR_INVALID_ARG),
    (dict(k_new=112, v_new=120), swa.SWA_ERR_INVALID_ARG),
    (dict(scale=float("nan")), swa.SWA_ERR_INVALID_ARG), (dict(sl=66), swa.SWA_ERR_INVALID_ARG),
    (dict(dims=(2, 513, 8, 2, 256, 4096, 0)), swa.SWA_ERR_INVALID_ARG),
    (dict(dims=(2, 8, 8, 2, 96, 4096, 0)), swa.SWA_ERR_UNSUPPORTED),
    (dict(paged=swa.SwaPaged(64, 256, 12, 600)), swa.SWA_ERR_INVALID_ARG),
    (dict(paged=swa.SwaPaged(None, 256, 16, 600)), swa.SWA_ERR_INVALID_ARG),
    (dict(paged=swa.SwaPaged(64, 255, 16, 600)), swa.SWA_ERR_INVALID_ARG),
])
def test_refusals(lib, kw, code):
    assert _call(lib, **kw) == code and swa.swa_last_error()


def test_binding_refuses_cpu_tensors():
    x = torch.zeros(1, 1, 2, 64, dtype=torch.bfloat16)
    i = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA device"):
        swa.swa_sink_verify_attn(x, x, x, i, i, 4, 1, 1.0)


def test_definition_without_sinks_is_the_windowed_oracle():
    rng = np.random.default_rng(0)
    q, k, v = (rng.standard_normal(s) for s in ((5, 4, 64), (2, 50, 64), (2, 50, 64)))
    out, lse, _, _ = vs.sink_attention(q, k, v, 45, 40, 7, 0, 0.1)
    ref_o, ref_l = oracle.attention(q[None], k[None], v[None], [45], [40], 7, 0.1)
    assert np.allclose(out, ref_o[0], atol=1e-13) and np.allclose(lse, ref_l[0], atol=1e-13)
    # sinks that cover the cache: full causal attention
    out, lse, _, _ = vs.sink_attention(q, k, v, 45, 40, 7, 64, 0.1)
    ref_o, ref_l = oracle.attention(q[None], k[None], v[None], [45], [40], 50, 0.1)
    assert np.allclose(out, ref_o[0], atol=1e-13) and np.allclose(lse, ref_l[0], atol=1e-13)
    # K = 0: the number of visible keys, sinks and window counted once
    for sinks, n in ((3, 10), (34, 41), (36, 41)):
        _, lse, _, _ = vs.sink_attention(q, 0 * k, v, 45, 40, 7, sinks, 0.1)
        assert np.allclose(lse[0], np.log(n))
