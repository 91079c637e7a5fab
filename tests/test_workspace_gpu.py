"""The library-owned workspaces on the GPU: what growing calls hold, and what
captured calls keep."""
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
