"""Sampled verification without a GPU: refusals of the C entry point before
any CUDA call, of the binding, and the definition's own invariants."""
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


PTRS = dict(logits=16, keep=32, draft=48, uniforms=64, temperature=80, top_k=96, top_p=112,
            min_p=128, tokens=144, logprobs=160, accepted=176)


def _call(lib, B=2, q_len=8, V=1000, sampling=True, **ptrs):
    p = {**PTRS, **ptrs}
    s = swa.SwaSampling(p["temperature"], p["top_k"], p["top_p"], p["min_p"])
    return lib.swa_sample_accept(p["logits"], p["keep"], p["draft"], p["uniforms"],
                                 ctypes.byref(s) if sampling else None, p["tokens"],
                                 p["logprobs"], p["accepted"], B, q_len, V, None)


@pytest.mark.parametrize("kw", [dict(B=0), dict(B=65536), dict(q_len=0), dict(q_len=65), dict(V=0),
                                dict(V=-5), dict(sampling=False)])
def test_bad_sizes(lib, kw):
    assert _call(lib, **kw) == swa.SWA_ERR_INVALID_ARG and swa.swa_last_error()


@pytest.mark.parametrize("name", ["logits", "draft", "uniforms", "temperature", "tokens",
                                  "accepted"])
def test_null_pointers(lib, name):
    assert _call(lib, **{name: None}) == swa.SWA_ERR_INVALID_ARG


@pytest.mark.parametrize("name", list(PTRS))
def test_misaligned_pointers(lib, name):
    assert _call(lib, **{name: PTRS[name] + 1}) == swa.SWA_ERR_INVALID_ARG
    assert "aligned" in swa.swa_last_error()


def test_binding_refusals():
    x = torch.zeros(1, 1, 8, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA device"):
        swa.swa_sample_accept(x, torch.zeros(1, 1), torch.ones(1))


def test_definition_against_plain_cases():
    x = np.array([1.0, 3.0, 2.0, 3.0, -np.inf, np.nan, 0.0])
    order = vs.sample_order(x)
    assert order.tolist() == [1, 3, 2, 0, 6]
    # u -> 0 is the argmax, as the greedy oracle has it
    assert vs.sample_row(x, 0.0, 1.0)[0] == 1 == vs.sample_row(x, 0.7, 0.0)[0]
    am, _ = oracle.greedy_accept(x.reshape(1, 1, -1), np.zeros((1, 0)))
    assert am[0, 0] == 1
    # every column's share of u is its softmax weight
    us = (np.arange(200000) + 0.5) / 200000
    w = vs.sample_weights(x, order, 0.7)
    cum = np.cumsum(w) / w.sum()
    got = [vs.sample_row(x, u, 0.7)[0] for u in us[::100]]
    assert got == [int(order[np.searchsorted(cum, u, side="right")]) for u in us[::100]]
    col, lp = vs.sample_row(x, 0.999, 1.0, top_k=3)
    assert col == 2 and abs(lp - np.log(np.exp(-1) / (2 + np.exp(-1)))) < 1e-15
    assert vs.sample_row(x, 0.999, 1.0, top_p=0.3)[0] == 1
    assert vs.sample_row(x, 0.999, 1.0, top_p=0.0) == (1, 0.0)
    assert vs.sample_row(x, 0.999, 1.0, min_p=0.5)[0] == 3
    assert vs.sample_row(np.array([-np.inf, np.nan]), 0.5, 1.0) == (0, 0.0)
    assert vs.accepted_prefix([[1, 2, 3], [1, 2, 3]], [[1, 5], [1, 2]]).tolist() == [1, 2]
