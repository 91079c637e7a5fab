"""Failures of the operators next to the attention, without a GPU fault: a
copy of the sink kernels that never lands (bounded waits run out and report),
launches that fail, and bad pages in the build with SWA_DEBUG_CHECKS."""
import json
import os
import subprocess
import sys

import pytest
import torch

from tests.helpers import forced_kernel
from tests.test_rope_gpu import _case
from tests.test_sink_gpu import Case

pytestmark = pytest.mark.gpu

LIMIT = 1_000_000       # SM cycles, about 0.5 ms
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import sliding_window_speculative_gb300 as swa
    from sliding_window_speculative_gb300 import build
    build.build()
    yield
    swa.swa_set_debug_options()


def _i32(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


def _args(c):
    """swa_sink_verify_attn's arguments and keywords for a test_sink_gpu.Case."""
    k, v, table, kn, vn = c.device()
    return ((c.q.cuda(), k, v, _i32(c.lens), _i32(c.pos), c.W, c.S, c.scale),
            dict(k_new=kn, v_new=vn, block_table=table))


# 147 key slots with 40 sinks (the first tile holds all of them), 235 with 128
# (a tensor-core tile of sinks alone): tensor-core fills 0 .. 3 are K and V of
# two tiles, the CUDA-core kernel's fills its 32-key tiles
@pytest.mark.parametrize("kernel,S,fill,page", [
    ("simt", 40, 0, 0),      # sinks
    ("simt", 40, 1, 16),     # the last sinks and the first window keys
    ("simt", 40, 4, 0),      # window keys
    ("tc", 40, 0, 0),        # K of the sinks' tile
    ("tc", 40, 3, 0),        # V of the window's last tile
    ("tc", 128, 1, 16),      # V of a tile of sinks alone
    ("rows", 40, 0, 16),
    ("rows", 128, 2, 0),     # K of the first tile without a sink
    ("rows", 40, 3, 0),
])
@pytest.mark.parametrize("batch", [1, 170])
def test_a_sink_copy_that_never_lands(kernel, S, fill, page, batch):
    import sliding_window_speculative_gb300 as swa
    c = Case(8, 8, 2, 128, 100, S, [300 + b % 50 for b in range(batch)], 512, page=page, seed=40)
    args, kw = _args(c)
    assert swa.swa_read_device_errors() == 0
    try:
        swa.swa_set_debug_options(force_kernel=kernel)
        want = swa.swa_sink_verify_attn(*args, **kw, num_splits=1)
        if batch == 1:
            c.check(*want, f"{kernel} before")
        swa.swa_set_debug_options(force_kernel=kernel, wait_limit_cycles=LIMIT, withhold_fill=fill)
        swa.swa_sink_verify_attn(*args, **kw, num_splits=1)
        torch.cuda.synchronize()                     # the call ended
        assert swa.swa_read_device_errors() & 1
        swa.swa_set_debug_options(force_kernel=kernel)
        again = swa.swa_sink_verify_attn(*args, **kw, num_splits=1)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(again, want))
        assert swa.swa_read_device_errors() == 0
    finally:
        swa.swa_set_debug_options()


@pytest.mark.parametrize("kernel,splits,nth,what", [
    ("simt", 1, 1, "attention kernel launch"), ("simt", 3, 2, "merge kernel launch"),
    ("tc", 1, 1, "tensor-core kernel launch"), ("tc", 3, 2, "merge kernel launch"),
    ("rows", 1, 1, "tensor-core kernel launch"), ("rows", 3, 2, "merge kernel launch"),
])
def test_sink_launch_failures(kernel, splits, nth, what):
    import sliding_window_speculative_gb300 as swa
    c = Case(8, 8, 2, 128, 200, 5, [300, 7], 512, seed=41)
    args, kw = _args(c)
    with forced_kernel(kernel):
        want = swa.swa_sink_verify_attn(*args, **kw, num_splits=splits)
        out, lse = (torch.full_like(t, 7.0) for t in want)
        swa.swa_set_debug_options(force_kernel=kernel, fail_launch=nth)
        with pytest.raises(swa.SwaError, match=what) as e:
            swa.swa_sink_verify_attn(*args, **kw, num_splits=splits, out=out, lse=lse)
        assert e.value.status == swa.SWA_ERR_CUDA
        assert swa.swa_get_debug_options()["fail_launch"] == 0
        torch.cuda.synchronize()
        assert (out == 7.0).all() and (lse == 7.0).all()
        again = swa.swa_sink_verify_attn(*args, **kw, num_splits=splits)
        torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(again, want))
    c.check(*again, f"{kernel} after a failed launch")


@pytest.mark.parametrize("kernel", ["simt", "tc", "rows"])
@pytest.mark.parametrize("page", [0, 16])
def test_a_failed_sink_append_leaves_the_cache(kernel, page):
    import sliding_window_speculative_gb300 as swa
    c = Case(8, 8, 2, 128, 60, 5, [300, 2], 512, page=page, append=True, seed=42)
    args, kw = _args(c)
    before = [t.clone() for t in args[1:3]]
    with forced_kernel(kernel):
        swa.swa_set_debug_options(force_kernel=kernel, fail_launch=1)
        with pytest.raises(swa.SwaError, match="launch"):
            swa.swa_sink_verify_attn(*args, **kw)
        torch.cuda.synchronize()
        for a, b in zip(args[1:3], before):
            assert torch.equal(a.view(torch.int16), b.view(torch.int16))
        c.check(*c.run(), f"{kernel} append after a failed launch")


@pytest.mark.parametrize("append", [False, True])
def test_rotation_launch_failures(append):
    import sliding_window_speculative_gb300 as swa
    c = _case(2, 5, 4, 2, 128, 64, seed=43, pos=[3, 20])
    k = torch.full((2, 2, 32, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    v, q_out = k.clone(), torch.full((2, 5, 4, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    rows = [torch.full((2, 5, 2, 128), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]

    def call():
        if append:
            pos = c["q_pos"]
            order = ("q", "k", "v", "q_weight", "k_weight", "eps", "inv_freq")
            swa.swa_qk_norm_rope_append(*(c[n] for n in order), k, v, pos + 5, pos, q_out=q_out)
            return [q_out, k, v]
        return list(swa.swa_qk_norm_rope(**c, q_out=q_out, k_out=rows[0], v_out=rows[1]))

    try:
        swa.swa_set_debug_options(fail_launch=1)
        with pytest.raises(swa.SwaError, match="rotation kernel launch") as e:
            call()
        assert e.value.status == swa.SWA_ERR_CUDA
    finally:
        swa.swa_set_debug_options()
    torch.cuda.synchronize()
    for t in [q_out, k, v] + rows:
        assert (t == 7.0).all()
    got = [t.clone() for t in call()]
    want = swa.swa_qk_norm_rope(**c)
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0])
    for t, w in zip(got[1:], want[1:]):
        if append:
            for b, p in enumerate((3, 20)):
                assert torch.equal(t[b, :, p:p + 5].transpose(0, 1), w[b])
                t[b, :, p:p + 5] = 7.0
            assert (t == 7.0).all()
        else:
            assert torch.equal(t, w)


# ---- the build with SWA_DEBUG_CHECKS, in a process of its own

@pytest.fixture(scope="module")
def debug_results():
    from sliding_window_speculative_gb300 import build
    build.build(debug_checks=True)
    r = subprocess.run([sys.executable, os.path.join(ROOT, "tests", "debug_checks_verify_step_run.py")],
                       capture_output=True, text=True, cwd=ROOT, timeout=600)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-3000:]
    lines = [json.loads(x) for x in r.stdout.splitlines() if x.startswith("{")]
    return {x["name"]: x for x in lines}


KERNELS = ("simt", "tc", "rows")


@pytest.mark.parametrize("name", ["rotation/valid"] + [f"{k}/valid" for k in KERNELS])
def test_debug_build_counts_nothing_on_valid_pages(debug_results, name):
    r = debug_results[name]
    assert r["ok"], r["detail"]
    assert r["count"] == 0


@pytest.mark.parametrize("name", ["rotation/bad page"] + [
    f"{k}/bad page of {what}" for k in KERNELS for what in ("the sinks", "the window", "the block")])
def test_debug_build_counts_and_contains_bad_pages(debug_results, name):
    r = debug_results[name]
    assert r["ok"], r["detail"]
    assert r["count"] > 0
