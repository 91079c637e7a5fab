"""The library-owned workspaces on the GPU: what growing calls hold, and what
captured calls keep."""
import os
import subprocess
import sys

import pytest
import torch

from sliding_window_speculative_gb300 import inputs
from tests.helpers import compare, oracle_reference, run_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sliding_window_speculative_gb300 import build
    build.build()
    yield


def _free():
    torch.cuda.synchronize()
    return torch.cuda.mem_get_info()[0]


def test_eager_calls_that_grow_hold_one_buffer():
    """Split calls of rising batch: afterwards the library holds the last one's
    buffer (a quarter more than it needs), not all of them."""
    import sliding_window_speculative_gb300 as swa
    swa.swa_release_workspace()
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    cases = [inputs.make_case("grow", B, 8, 2, 256, 64, 2048, [4096] * B, 4096, seed=B, device="cuda")
             for B in (4, 6, 9)]
    need = [swa.swa_plan(swa.dims_of(c.q, c.k_cache, 16), c.window, sms)["workspace_bytes"]
            for c in cases]
    assert all(b > a > 32 << 20 for a, b in zip(need, need[1:]))
    for c in cases:             # (anything else a first call allocates)
        run_gpu(c, 1)
    outs = [(torch.empty_like(c.q), torch.empty(c.q.shape[:3], device="cuda")) for c in cases]
    before = _free()
    for c, (out, lse) in zip(cases, outs):
        swa.swa_verify_attn(c.q, c.k_cache, c.v_cache, c.seq_lens, c.q_pos, c.window, c.scale,
                            out=out, lse=lse, num_splits=16)
    held = before - _free()
    assert held <= need[-1] * 5 // 4 + (8 << 20), (held, need)
    for c, (out, lse) in zip(cases, outs):
        compare(out, lse, *oracle_reference(c), f"split call of {c.q.shape[0]}")
    swa.swa_release_workspace()
    assert before - _free() <= 4 << 20


CAPTURED_ACCEPT = r"""
import torch
import sliding_window_speculative_gb300 as swa

g = torch.Generator().manual_seed(3)
logits = torch.randn((2, 8, 5000), generator=g).to(torch.bfloat16).cuda()
draft = torch.randint(0, 5000, (2, 7), generator=g, dtype=torch.int32).cuda()
want = [t.clone() for t in swa.swa_greedy_accept(logits, draft)]
draft[:, :5] = want[0][:, :5]
want = [t.clone() for t in swa.swa_greedy_accept(logits, draft)]
am, acc = torch.zeros_like(want[0]), torch.zeros_like(want[1])
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    swa.swa_greedy_accept(logits, draft, argmax=am, accepted=acc)
big = torch.zeros((65535, 64, 1), dtype=torch.bfloat16, device="cuda")
bd = torch.zeros((65535, 63), dtype=torch.int32, device="cuda")
bm, bc = swa.swa_greedy_accept(big, bd)                  # outgrows the graph's scratch
filler = torch.full((1 << 22,), -1, dtype=torch.int32, device="cuda")
for _ in range(3):
    am.zero_(), acc.zero_()
    graph.replay()
    again = swa.swa_greedy_accept(logits, draft)          # and an eager call beside it
    torch.cuda.synchronize()
    assert torch.equal(am, want[0]) and torch.equal(acc, want[1])
    assert all(torch.equal(a, b) for a, b in zip(again, want))
assert not bm.any() and (bc == 63).all() and (filler == -1).all()
print("ok")
"""


def test_a_captured_acceptance_survives_a_larger_call():
    """In a process of its own: the scratch has to be outgrown after the capture."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", CAPTURED_ACCEPT], capture_output=True, text=True,
                       cwd=root, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr[-2000:]
