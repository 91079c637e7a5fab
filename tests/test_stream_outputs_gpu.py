"""Outputs that the binding allocates for a call on another stream than the
current one: never memory that the current stream may still be using, and not
given away while either stream is."""
import pytest
import torch

pytestmark = pytest.mark.gpu

B, Q, HQ, HKV, D, L, V = 4, 8, 8, 2, 128, 256, 16384


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sliding_window_speculative_gb300 import build
    build.build()
    yield


def _calls():
    """name -> f(stream) giving the call's allocated outputs."""
    import sliding_window_speculative_gb300 as swa
    g = torch.Generator().manual_seed(8)
    rnd = lambda *s: torch.randn(s, generator=g).to(torch.bfloat16).cuda()  # noqa: E731
    q, kn, vn = rnd(B, Q, HQ, D), rnd(B, Q, HKV, D), rnd(B, Q, HKV, D)
    k, v = rnd(B, HKV, L, D), rnd(B, HKV, L, D)
    kp, vp = rnd(B * L // 16, HKV, 16, D), rnd(B * L // 16, HKV, 16, D)
    table = torch.arange(B * L // 16, dtype=torch.int32).view(B, L // 16).cuda()
    pos = torch.tensor([0, 9, 100, 248], dtype=torch.int32).cuda()
    lens = pos + Q
    f = torch.logspace(0, -4, D // 2).cuda()
    x, u, T = rnd(B, Q, V), torch.rand((B, Q), generator=g).cuda(), torch.ones(B).cuda()
    draft = torch.zeros((B, Q - 1), dtype=torch.int32).cuda()
    s = D ** -0.5
    return {
        "swa_verify_attn": lambda st: swa.swa_verify_attn(q, k, v, lens, pos, 50, s, stream=st),
        "swa_verify_attn_paged": lambda st: swa.swa_verify_attn_paged(
            q, kp, vp, table, lens, pos, 50, s, stream=st),
        "swa_append_verify_attn": lambda st: swa.swa_append_verify_attn(
            q, kn, vn, k, v, lens, pos, 50, s, stream=st),
        "swa_sink_verify_attn": lambda st: swa.swa_sink_verify_attn(
            q, k, v, lens, pos, 50, 4, s, stream=st),
        "swa_qk_norm_rope": lambda st: swa.swa_qk_norm_rope(
            q, kn, vn, None, None, 1e-6, f, pos, stream=st),
        "swa_qk_norm_rope_append": lambda st: (swa.swa_qk_norm_rope_append(
            q, kn, vn, None, None, 1e-6, f, k, v, lens, pos, stream=st),),
        "swa_sample_accept": lambda st: swa.swa_sample_accept(x, u, T, draft=draft, stream=st),
        "swa_greedy_accept": lambda st: swa.swa_greedy_accept(x, draft, stream=st),
    }


NAMES = ("swa_verify_attn", "swa_verify_attn_paged", "swa_append_verify_attn",
         "swa_sink_verify_attn", "swa_qk_norm_rope", "swa_qk_norm_rope_append",
         "swa_sample_accept", "swa_greedy_accept")


@pytest.fixture(scope="module")
def calls():
    c = _calls()
    assert tuple(c) == NAMES
    for f in c.values():
        f(None)
    torch.cuda.synchronize()
    return c


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("as_handle", [False, True])
def test_outputs_are_not_the_current_streams_memory(calls, name, as_handle):
    """Blocks just freed on the current stream, of every output's size, are not
    what the outputs get."""
    side = torch.cuda.Stream()
    stream = side.cuda_stream if as_handle else side
    want = [t.clone() for t in calls[name](None)]
    torch.cuda.synchronize()
    side.wait_stream(torch.cuda.current_stream())
    freed = [torch.empty_like(t) for t in want for _ in range(4)]
    blocks = {t.data_ptr() for t in freed}
    del freed
    got = calls[name](stream)
    assert not blocks & {t.data_ptr() for t in got}
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("name", NAMES)
def test_freed_outputs_wait_for_the_current_stream(calls, name):
    """Results read late on the current stream and freed at once: the next call
    on the side stream leaves them alone."""
    side = torch.cuda.Stream()
    here = torch.cuda.current_stream()
    want = [t.clone() for t in calls[name](None)]
    torch.cuda.synchronize()
    got = calls[name](side)
    blocks = {t.data_ptr() for t in got}
    here.wait_stream(side)
    torch.cuda._sleep(20_000_000)        # about 10 ms
    late = [t.clone() for t in got]
    del got
    again = calls[name](side)
    assert not blocks & {t.data_ptr() for t in again}
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(late, want))
    assert all(torch.equal(a, b) for a, b in zip(again, want))


@pytest.mark.parametrize("name", NAMES)
def test_the_current_stream_by_handle(calls, name):
    want = [t.clone() for t in calls[name](None)]
    got = calls[name](torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
