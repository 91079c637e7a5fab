"""A program whose very first call of an operator is captured: nothing of the
operators next to the attention needs a call before the capture (but split
partials, which are refused with a message)."""
import os
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

COMMON = r"""
import torch
import sliding_window_speculative_gb300 as swa
g = torch.Generator().manual_seed(5)
rnd = lambda *s: torch.randn(s, generator=g).to(torch.bfloat16).cuda()
i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()
pos, lens = i32([3, 700]), i32([11, 708])
def check(call):
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call()
    graph.replay()
    want = call()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    print("ok")
"""

CALLS = {
    "sink": """
q, k, v = rnd(2, 8, 8, 256), rnd(2, 2, 1024, 256), rnd(2, 2, 1024, 256)
check(lambda: swa.swa_sink_verify_attn(q, k, v, lens, pos, 188, 4, 1 / 16))
""",
    "rope": """
x, f = rnd(2, 8, 12, 256), torch.logspace(0, -4, 128).cuda()
w = torch.ones(256).cuda()
check(lambda: swa.swa_qk_norm_rope(x[:, :, :8], x[:, :, 8:10], x[:, :, 10:], w, w, 1e-6, f, pos))
""",
    "rope_append": """
x, f = rnd(2, 8, 12, 256), torch.logspace(0, -4, 128).cuda()
k, v = rnd(2, 2, 1024, 256), rnd(2, 2, 1024, 256)
check(lambda: (swa.swa_qk_norm_rope_append(x[:, :, :8], x[:, :, 8:10], x[:, :, 10:], None, None, 1e-6,
                                           f, k, v, lens, pos), k, v))
""",
    "sample": """
x, u, T = rnd(2, 8, 50001), torch.rand((2, 8), generator=g).cuda(), torch.ones(2).cuda()
draft = torch.zeros((2, 7), dtype=torch.int32).cuda()
check(lambda: swa.swa_sample_accept(x, u, T, draft=draft))
""",
    "sink_splits": """
q, k, v = rnd(2, 8, 8, 256), rnd(2, 2, 1024, 256), rnd(2, 2, 1024, 256)
call = lambda: swa.swa_sink_verify_attn(q, k, v, lens, pos, 600, 4, 1 / 16, num_splits=3)
graph = torch.cuda.CUDAGraph()
y = torch.zeros(8, device="cuda")
with torch.cuda.graph(graph):
    y += 1
    try:
        call()
        raise AssertionError("not refused")
    except swa.SwaError as e:
        assert e.status == swa.SWA_ERR_WORKSPACE, e
graph.replay()
torch.cuda.synchronize()
assert (y == 1).all()
call()
check(call)
""",
}


@pytest.mark.parametrize("name", CALLS)
def test_first_call_in_a_capture(name):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sliding_window_speculative_gb300 import build
    build.build()
    r = subprocess.run([sys.executable, "-c", COMMON + CALLS[name]], capture_output=True, text=True,
                       cwd=ROOT, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr[-2000:]
