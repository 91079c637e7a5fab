"""The 8-bit cache and the token log probabilities as a server uses them: together,
captured and replayed, on other streams, in one workspace, with copies that never
land, launches that fail and caches past 2^32 bytes.

The attention is compared with the 64-bit definition over the rows read back, within
the bounds of tests/test_q8_gpu.py; everything that runs twice has to give the same
bits."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import oracle.kv8 as kv8
from tests.helpers import forced_kernel

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
E4M3 = torch.float8_e4m3fn
KERNELS = ["plan", "tc", "rows"]


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sliding_window_speculative_gb300 import build
    build.build()
    yield
    import sliding_window_speculative_gb300 as swa
    swa.swa_set_debug_options()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def empty_cache(B, Hkv, L, D, page=0):
    shape = (B * (L // page), Hkv, page) if page else (B, Hkv, L)
    table = None
    if page:
        g = torch.Generator().manual_seed(L)
        table = torch.randperm(shape[0], generator=g).view(B, -1).to(torch.int32).cuda()
    data = [torch.zeros((*shape, D), dtype=torch.uint8, device="cuda").view(E4M3) for _ in range(2)]
    return [*data, *(torch.zeros(shape, dtype=torch.int8, device="cuda") for _ in range(2))], table


def check_attention(q, k, v, lens, pos, W, out, lse):
    """out and lse [B, q, Hq, ..] against the definition over values k, v
    [B, Hkv, L, D]; the bounds of tests/test_q8_gpu.py."""
    D = q.shape[-1]
    for b in range(q.shape[0]):
        o, z, mag, wv, seen = kv8.attention(q[b].double().cpu().numpy(), k[b], v[b], lens[b], pos[b],
                                            W, D ** -0.5)
        d = (D + 16) * 2.0 ** -24 * mag + 2.0 ** -20
        tol = (2.0 ** -8 * np.abs(o) + (2 * d + 2.0 ** -8)[..., None] * wv +
               (seen * 2.0 ** -20)[..., None] * np.abs(v[b]).max())
        assert np.all(np.abs(out[b].double().cpu().numpy() - o) <= tol), b
        ez = np.abs(lse[b].double().cpu().numpy() - z)
        assert np.all(ez <= d + 2.0 ** -20 + 2.0 ** -22 * np.abs(z)), b


# ---------------------------------------------------------------- together

@pytest.mark.parametrize("D,page", [(256, 0), (256, 16), (128, 8), (64, 0)])
def test_a_serving_loop_captured_and_replayed(D, page):
    """Prefill, then verify steps: normalise and rotate, append, attend, sample and
    report; the steps as one captured graph give what eager calls give."""
    import sliding_window_speculative_gb300 as swa
    B, q_len, Hq, Hkv, L, W, V, T0 = 3, 4, 8, 2, 256, 100, 500, 90
    g = torch.Generator(device="cuda").manual_seed(D + page)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    f = torch.logspace(0, -4, D // 2).cuda()
    w = torch.ones(D).cuda()
    temp = torch.tensor([0.7, 1.0, 0.0]).cuda()
    prompt = rnd(B, T0, Hq + 2 * Hkv, D)
    start = [T0, T0 - 31, T0 - 89]                 # the prompts' lengths; the last has one token
    steps = [rnd(B, q_len, Hq + 2 * Hkv, D) for _ in range(5)]
    u = torch.rand((5, B, q_len), generator=g, device="cuda")
    draft = torch.randint(0, V, (5, B, q_len - 1), generator=g, device="cuda").to(torch.int32)

    def project(x, pos):
        q, k, v = x.split([Hq, Hkv, Hkv], dim=2)
        return swa.swa_qk_norm_rope(q, k, v, w, w, 1e-6, f, pos)

    def step(cache, table, x, uu, dd, pos, lens):
        q, k, v = project(x, pos)
        swa.swa_q8_append(k, v, *cache, lens, pos, block_table=table)
        out, lse = swa.swa_q8_verify_attn(q, *cache, lens, pos, W, D ** -0.5, block_table=table)
        logits = (out.reshape(B, q_len, Hq * D)[..., :V] * 8).contiguous()
        res = swa.swa_sample_accept(logits, uu, temp, draft=dd)
        lp = swa.swa_token_logprobs(logits, res[0], top_n=5, temperature=temp)
        return [q, out, lse, logits, *res, *lp]

    def prefill(cache, table):
        pos = i32([0] * B)
        q, k, v = project(prompt, pos)
        swa.swa_q8_append(k, v, *cache, i32(start), pos, block_table=table)

    # eager
    cache, table = empty_cache(B, Hkv, L, D, page)
    prefill(cache, table)
    want = []
    for t in range(5):
        pos = i32([n + q_len * t for n in start])
        lens = pos + q_len
        got = step(cache, table, steps[t], u[t], draft[t], pos, lens)
        want.append([None if x is None else x.clone() for x in got])
        k, v = swa.swa_q8_read(*cache, lens, i32([0] * B), L, block_table=table)
        check_attention(got[0], k.double().cpu().numpy(), v.double().cpu().numpy(), lens.tolist(),
                        pos.tolist(), W, got[1], got[2])
    # captured: one step with its inputs in fixed buffers, on a side stream
    cache2, table2 = empty_cache(B, Hkv, L, D, page)
    if page:
        assert torch.equal(table, table2)
    prefill(cache2, table2)
    x, uu, dd = steps[0].clone(), u[0].clone(), draft[0].clone()
    pos = i32(start)
    lens = pos + q_len
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got = step(cache2, table2, x, uu, dd, pos, lens)
        pos += q_len
        lens += q_len
    for t in range(5):
        x.copy_(steps[t])
        uu.copy_(u[t])
        dd.copy_(draft[t])
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want[t]):
            assert (a is None) == (b is None)
            if a is not None:
                # (as bits: an entropy or a logit of no token may be NaN or infinite)
                assert torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))
    for a, b in zip(cache, cache2):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    assert swa.swa_read_device_errors() == 0


# ------------------------------------------------------------------ streams

def _calls():
    """name -> f(stream) giving the call's allocated outputs."""
    import sliding_window_speculative_gb300 as swa
    B, Q, Hq, Hkv, L, V = 4, 8, 8, 2, 256, 16384
    g = torch.Generator(device="cuda").manual_seed(8)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    pos = i32([0, 9, 100, 248])
    lens, zero = pos + Q, i32([0] * B)
    made = {}
    for D in (128, 256):
        cache, table = empty_cache(B, Hkv, L, D, 16 if D == 256 else 0)
        swa.swa_q8_append(rnd(B, L, Hkv, D), rnd(B, L, Hkv, D), *cache, zero + L, zero,
                          block_table=table)
        made[D] = (cache, table, rnd(B, Q, Hq, D), rnd(B, 200, Hq, D))
    x, tok = rnd(B, Q, V), torch.randint(0, V, (B, Q), generator=g, device="cuda").to(torch.int32)

    def attend(D, long, splits=0):
        cache, table, q, q_long = made[D]
        return lambda st: swa.swa_q8_verify_attn(
            q_long if long else q, *cache, zero + L if long else lens, zero if long else pos, 150,
            D ** -0.5, block_table=table, num_splits=splits, stream=st)

    return {
        "read": lambda st: swa.swa_q8_read(*made[128][0], lens, pos, 20, stream=st),
        "read_paged": lambda st: swa.swa_q8_read(*made[256][0], lens, pos, 20,
                                                 block_table=made[256][1], stream=st),
        "attn": attend(128, False),
        "attn_paged": attend(256, False),
        "attn_splits": attend(256, False, 3),
        "attn_rows": attend(128, True),
        "logprobs": lambda st: swa.swa_token_logprobs(x, tok, top_n=7, stream=st),
    }


NAMES = ("read", "read_paged", "attn", "attn_paged", "attn_splits", "attn_rows", "logprobs")


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


def test_two_graphs_in_one_workspace(calls):
    """Captured calls with split partials or bf16 rows in the workspace, replayed in
    turn on one stream."""
    names = ("attn_splits", "attn_rows", "attn")
    want = {n: [t.clone() for t in calls[n](None)] for n in names}
    torch.cuda.synchronize()
    graphs = {}
    for n in names:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = calls[n](None)
        graphs[n] = (graph, got)
    for _ in range(3):
        for n in names:
            for t in graphs[n][1]:
                t.zero_()
            graphs[n][0].replay()
        torch.cuda.synchronize()
        for n in names:
            assert all(torch.equal(a, b) for a, b in zip(graphs[n][1], want[n])), n


# ----------------------------------------------------- a first captured call

FIRST = r"""
import torch
import sliding_window_speculative_gb300 as swa
g = torch.Generator(device="cuda").manual_seed(5)
rnd = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)
i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()
pos, lens = i32([3, 700]), i32([11, 708])
cache = [torch.zeros((2, 2, 1024, 256), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
         for _ in range(2)] + [torch.zeros((2, 2, 1024), dtype=torch.int8, device="cuda") for _ in range(2)]
k, v, q = rnd(2, 8, 2, 256), rnd(2, 8, 2, 256), rnd(2, 8, 8, 256)
def check(call):
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call()
    graph.replay()
    want = call()
    torch.cuda.synchronize()
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(got, want))
    print("ok")
"""

FIRST_CALLS = {
    "append": "check(lambda: swa.swa_q8_append(k, v, *cache, lens, pos))",
    "read": "check(lambda: swa.swa_q8_read(*cache, lens, pos, 9))",
    "attn": "check(lambda: swa.swa_q8_verify_attn(q, *cache, lens, pos, 188, 1 / 16))",
    "logprobs": """
x, tok = rnd(2, 8, 50001), i32([[5] * 8] * 2)
check(lambda: swa.swa_token_logprobs(x, tok, top_n=3))
""",
    "splits": """
call = lambda: swa.swa_q8_verify_attn(q, *cache, lens, pos, 600, 1 / 16, num_splits=3)
graph = torch.cuda.CUDAGraph()
y = torch.zeros(8, device="cuda")
with torch.cuda.graph(graph):
    y += 1
    try:
        call()
        raise SystemExit("not refused")
    except swa.SwaError as e:
        assert e.status == swa.SWA_ERR_WORKSPACE and "capture" in str(e), str(e)
graph.replay()
torch.cuda.synchronize()
assert float(y.sum()) == 8
swa.swa_set_workspace(torch.empty(swa.swa_q8_workspace_bytes(swa.dims_of(q, cache[0], 3), 600),
                                  dtype=torch.uint8, device="cuda"))
check(call)
""",
}


@pytest.mark.parametrize("name", list(FIRST_CALLS))
def test_first_call_is_captured(name):
    r = subprocess.run([sys.executable, "-c", FIRST + FIRST_CALLS[name]], capture_output=True,
                       text=True, cwd=ROOT, timeout=600)
    assert r.returncode == 0 and r.stdout.strip().endswith("ok"), r.stderr[-2000:]


# ------------------------------------------------- waits that run out, launches

def _case(B, D, W, q_len=8, page=0, seed=0):
    """(q, cache, table, lens, pos): B sequences of 300 positions and more."""
    import sliding_window_speculative_gb300 as swa
    Hq, Hkv, L = 8, 2, 512
    cache, table = empty_cache(B, Hkv, L, D, page)
    g = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    zero = i32([0] * B)
    swa.swa_q8_append(rnd(B, L, Hkv, D), rnd(B, L, Hkv, D), *cache, zero + L, zero, block_table=table)
    lens = i32([300 + (37 * b) % 200 for b in range(B)])
    return rnd(B, q_len, Hq, D), cache, table, lens, lens - q_len


@pytest.mark.parametrize("B,D,page,fill,splits", [
    (1, 256, 0, 0, 0),      # K of the first tile
    (1, 256, 0, 1, 0),      # V of the first tile
    (1, 128, 0, 2, 0),      # K of the second tile
    (1, 128, 16, 3, 0),     # the last V tile, of pages
    (1, 256, 16, 0, 3),     # a split plan
    (200, 256, 0, 5, 0),    # mid-item, several items per CTA
    (200, 128, 8, 6, 0),
])
def test_withheld_copy_runs_out_and_reports(B, D, page, fill, splits):
    """A copy that is never issued: the call ends, the device word says so, the next
    call is right."""
    import sliding_window_speculative_gb300 as swa
    q, cache, table, lens, pos = _case(B, D, 188, page=page)
    call = lambda: swa.swa_q8_verify_attn(q, *cache, lens, pos, 188, D ** -0.5,  # noqa: E731
                                          block_table=table, num_splits=splits)
    want = [t.clone() for t in call()]
    torch.cuda.synchronize()
    assert swa.swa_read_device_errors() == 0
    try:
        swa.swa_set_debug_options(wait_limit_cycles=1_000_000, withhold_fill=fill)
        call()
        torch.cuda.synchronize()
        assert swa.swa_read_device_errors() & 1
    finally:
        swa.swa_set_debug_options()
    got = call()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert swa.swa_read_device_errors() == 0


@pytest.mark.parametrize("name,kernel,splits,nth,what", [
    ("append", "plan", 0, 1, "8-bit append kernel launch"),
    ("read", "plan", 0, 1, "8-bit read kernel launch"),
    ("attn", "tc", 0, 1, "8-bit attention kernel launch"),
    ("attn", "tc", 3, 2, "merge kernel launch"),
    ("attn", "rows", 0, 1, "8-bit window kernel launch"),
    ("attn", "rows", 0, 2, "tensor-core kernel launch"),
    ("attn", "rows", 3, 3, "merge kernel launch"),
    ("logprobs", "plan", 0, 1, "log probability kernel launch"),
])
def test_injected_launch_failure(name, kernel, splits, nth, what):
    """A launch that fails: the error names it, no output is written, the next call is
    right."""
    import sliding_window_speculative_gb300 as swa
    q, cache, table, lens, pos = _case(2, 256, 188)
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn((2, 3, 5000), generator=g, device="cuda").to(torch.bfloat16)
    tok = torch.randint(0, 5000, (2, 3), generator=g, device="cuda").to(torch.int32)
    new = torch.randn((2, 8, 2, 256), generator=g, device="cuda").to(torch.bfloat16)
    outs = {
        "append": lambda: [t.clone() for t in cache],
        "read": lambda: [torch.full((2, 2, 9, 256), 7.0, dtype=torch.bfloat16, device="cuda")
                         for _ in range(2)],
        "attn": lambda: [torch.full_like(q, 7.0), torch.full(q.shape[:3], 7.0, device="cuda")],
        "logprobs": lambda: [torch.full((2, 3), 7.0, device="cuda")],
    }[name]
    call = {
        "append": lambda o: swa.swa_q8_append(new, new, *o, lens, pos),
        "read": lambda o: swa.swa_q8_read(*cache, lens, pos, 9, k_out=o[0], v_out=o[1]),
        "attn": lambda o: swa.swa_q8_verify_attn(q, *cache, lens, pos, 188, 1 / 16, out=o[0],
                                                 lse=o[1], num_splits=splits),
        "logprobs": lambda o: swa.swa_token_logprobs(x, tok, logprobs=o[0]),
    }[name]
    with forced_kernel(kernel):
        want = outs()
        call(want)
        torch.cuda.synchronize()
        o = outs()
        before = [t.clone() for t in o]
        try:
            swa.swa_set_debug_options(force_kernel=0 if kernel == "plan" else kernel, fail_launch=nth)
            with pytest.raises(swa.SwaError) as e:
                call(o)
        finally:
            swa.swa_set_debug_options()
    assert e.value.status == swa.SWA_ERR_CUDA and what in str(e.value), str(e.value)
    torch.cuda.synchronize()
    bits = lambda t: t.view(torch.uint8)  # noqa: E731
    assert all(torch.equal(bits(a), bits(b)) for a, b in zip(o, before))
    with forced_kernel(kernel):
        call(o)
        torch.cuda.synchronize()
    assert all(torch.equal(bits(a), bits(b)) for a, b in zip(o, want))


# ------------------------------------------------------------- long caches

@pytest.mark.parametrize("paged", [False, True])
def test_offsets_past_32_bits(paged):
    """A cache tensor of more than 2^32 bytes, its last positions (or pages) used."""
    import sliding_window_speculative_gb300 as swa
    D, q_len, W, Hq = 256, 8, 188, 4
    L = (1 << 24) + 512                       # rows of 256 bytes
    if torch.cuda.mem_get_info()[0] < 12 << 30:
        pytest.skip("needs 12 GB")
    page = 16
    shape = (L // page, 1, page) if paged else (1, 1, L)
    cache = [torch.zeros((*shape, D), dtype=torch.uint8, device="cuda").view(E4M3) for _ in range(2)]
    cache += [torch.zeros(shape, dtype=torch.int8, device="cuda") for _ in range(2)]
    n, ctx = 512, (512 if paged else L)
    table = None
    if paged:                                 # the pool's last pages, in falling order
        table = (L // page - 1 - torch.arange(n // page)).to(torch.int32).view(1, -1).cuda()
    g = torch.Generator(device="cuda").manual_seed(1)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    k, v, q = rnd(1, n, 1, D), rnd(1, n, 1, D), rnd(1, q_len, Hq, D)
    lens, pos = i32([ctx]), i32([ctx - n])
    swa.swa_q8_append(k, v, *cache, lens, pos, block_table=table)
    kr, vr = swa.swa_q8_read(*cache, lens, pos, n, block_table=table)
    for x, y in ((k, kr), (v, vr)):
        x, y = x[0, :, 0].double(), y[0, 0].double()
        step = 2.0 ** (torch.ceil(torch.log2(x.abs().amax(dim=-1, keepdim=True) / 448)) - 10)
        assert ((y - x).abs() <= torch.maximum(2.0 ** -4 * x.abs(), step * (1 + 2.0 ** -40))).all()
    # nothing was written anywhere else
    assert int(sum((c.view(torch.uint8).view(-1, D)[:, :8] != 0).any(dim=1).sum() for c in cache[:1])) <= n
    for kernel in KERNELS:
        with forced_kernel(kernel):
            out, lse = swa.swa_q8_verify_attn(q, *cache, lens, lens - q_len, W, 1 / 16,
                                              block_table=table)
        torch.cuda.synchronize()
        check_attention(q, kr.double().cpu().numpy(), vr.double().cpu().numpy(), [n], [n - q_len], W,
                        out, lse)
    assert swa.swa_read_device_errors() == 0


# --------------------------------------------------------------- workloads

def test_workloads_agree():
    """The workloads of perf/more_operators.py: their plain forms, the library's calls
    and their 64-bit definitions, on the smaller listed cases and on drawn ones."""
    import random

    import perf.more_operators as M
    rng = random.Random(11)
    drawn = [M.draw(rng) for _ in range(80)]
    cases = [c for c in M.listed() if M.work(c)["bytes"] < 1e7]
    cases += [c for c in drawn if M.work(c)["bytes"] < 2e7][:20]
    assert {c["op"] for c in cases} == {"cache", "attn", "logprobs"} and len(cases) > 18
    compared = 0
    for n, case in enumerate(cases):
        want = M.exact(dict(case), 200 + n)
        if want is None:
            continue
        compared += 1
        for own in (False, True):
            M.own = own
            try:
                st = M.prepare(dict(case), 200 + n)
                got = M.run(st)
                torch.cuda.synchronize()
            finally:
                M.own = False
            for i, (a, w) in enumerate(zip(got, want)):
                if w is None:
                    continue
                what = (case, own, i)
                if case["op"] == "cache" or not a.dtype.is_floating_point:
                    # whole numbers, and values that are bf16 or e4m3 numbers; the
                    # definition's powers of two are a 64-bit pow(), within 2 units in
                    # the last place (2^-51), and their products round once more
                    x, y = kv8_values(a), w.double()
                    same = (x - y).abs() <= 2.0 ** -50 * y.abs()
                    assert (same | (x.isnan() & y.isnan())).all(), what
                    continue
                a, w = a.double(), w.double()
                inf = torch.isinf(w)
                assert torch.equal(a[inf], w[inf]), what
                if case["op"] == "attn":
                    # by |q||k| and the largest |v|; see tests/test_q8_gpu.py
                    q2 = st["q"].double().square().sum(-1).amax().sqrt()
                    k = kv8_values(st["k_cache"]) * 2.0 ** st["k_exp"].double()[..., None]
                    v = kv8_values(st["v_cache"]) * 2.0 ** st["v_exp"].double()[..., None]
                    mag = case["D"] ** -0.5 * q2 * k.square().sum(-1).amax().sqrt()
                    d = (case["D"] + 16) * 2.0 ** -24 * mag + 2.0 ** -20
                    tol = (2.0 ** -8 * w.abs() + (2 * d + 2.0 ** -8 + 2.0 ** -20 * case["W"]) *
                           v.abs().amax() if i == 0 else d + 2.0 ** -20 + 2.0 ** -22 * w.abs())
                else:
                    base = (case["V"] / 32 + 64) * 2.0 ** -24 + 2.0 ** -20
                    tol = (base + 2.0 ** -22) * (1 + 2 * w.abs())
                assert ((a - w).abs() <= tol)[~inf].all(), what
        del st, got, want
        torch.cuda.empty_cache()
    assert compared > 12


def kv8_values(t):
    if t.dtype == E4M3:
        table = torch.from_numpy(kv8.E4M3).cuda()
        return table[t.view(torch.uint8).long()]
    return t.double()
