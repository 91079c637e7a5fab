"""Child process of tests/test_verify_step_failures_gpu.py: the library built
with SWA_DEBUG_CHECKS on the sink attention and the rotation into pages.
Prints one JSON line per case: {"name", "count", "ok", "detail"}.

A bad page is one past the pool that the call is given, in guard pages that
the test owns, filled with marker values: even an unchecked access would stay
in the test's memory and show."""
import json
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import torch  # noqa: E402

from sliding_window_speculative_gb300 import _binding  # noqa: E402

_binding.load_library(_binding.DEBUG_LIB_PATH)

import sliding_window_speculative_gb300 as swa  # noqa: E402
from tests.test_rope_gpu import _case  # noqa: E402
from tests.test_sink_gpu import Case  # noqa: E402

MARK = 1000.0
PAGE, L = 16, 512


def record(name, fn):
    swa.swa_read_debug_checks()
    try:
        fn()
        ok, detail = True, ""
    except Exception as e:  # reported to the parent test
        ok, detail = False, repr(e)[:400]
    print(json.dumps({"name": name, "count": swa.swa_read_debug_checks(), "ok": ok,
                      "detail": detail}), flush=True)


def i32(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


def guarded(pool):
    """The pool with three marked pages behind it."""
    g = torch.full((3,) + tuple(pool.shape[1:]), MARK, dtype=pool.dtype, device="cuda")
    return torch.cat([pool, g])


def sink_call(c, bad=None):
    """One call; block `bad` of sequence 0 is a page past the pool."""
    k, v, table, kn, vn = c.device()
    # (page 0 is read in place of a bad one: nothing there may be NaN)
    n = k.shape[0]
    k, v = (guarded(torch.nan_to_num(t, nan=0.5)) for t in (k, v))
    good = table.clone()
    if bad is not None:
        table[0, bad] = n + 1
    k0, v0 = k.clone(), v.clone()
    out, lse = swa.swa_sink_verify_attn(c.q.cuda(), k[:n], v[:n], i32(c.lens), i32(c.pos), c.W, c.S,
                                        c.scale, k_new=kn, v_new=vn, block_table=table)
    torch.cuda.synchronize()
    assert (k[n:] == MARK).all() and (v[n:] == MARK).all(), "a guard page was written"
    for t, t0, new in ((k, k0, kn), (v, v0, vn)):
        for b, p in enumerate(c.pos):
            for i in range(c.q.shape[1]):
                j = p + i
                if b == 0 and j // PAGE == bad:
                    continue                     # dropped
                t0[int(good[b, j // PAGE]), :, j % PAGE] = new[b, i]
        assert torch.equal(t, t0), "another row than the block's was written"
    return out, lse


def sinks(kernel):
    swa.swa_set_debug_options(force_kernel=kernel)
    c = Case(8, 8, 2, 128, 60, 20, [300, 100], L, page=PAGE, append=True, seed=50)
    want = []

    def valid():
        want.extend(sink_call(c))
        c.check(*want, kernel)
    record(f"{kernel}/valid", valid)
    for what, block in (("the sinks", 1), ("the window", 260 // PAGE), ("the block", 300 // PAGE)):
        def bad():
            out, lse = sink_call(c, block)
            assert torch.isfinite(out).all() and out[0].float().abs().max() < 100, "a guard page was read"
            assert torch.equal(out[1], want[0][1]) and torch.equal(lse[1], want[1][1])
        record(f"{kernel}/bad page of {what}", bad)


def rotation():
    swa.swa_set_debug_options()
    c = _case(2, 20, 4, 2, 128, 128, seed=51, pos=[3, 100])
    pos = c["q_pos"]
    nb = 10
    pool = torch.full((2 * nb, 2, PAGE, 128), 0.5, dtype=torch.bfloat16, device="cuda")
    k0, v0 = guarded(pool), guarded(pool)
    rows = swa.swa_qk_norm_rope(**c)
    order = ("q", "k", "v", "q_weight", "k_weight", "eps", "inv_freq")

    def call(bad):
        table = torch.arange(2 * nb, dtype=torch.int32).view(2, nb)
        k, v, kw, vw = k0.clone(), v0.clone(), k0.clone(), v0.clone()
        for b, p in enumerate((3, 100)):
            for i in range(20):
                j = p + i
                if (b, j // PAGE) != bad:
                    kw[int(table[b, j // PAGE]), :, j % PAGE] = rows[1][b, i]
                    vw[int(table[b, j // PAGE]), :, j % PAGE] = rows[2][b, i]
        if bad:
            table[bad] = 2 * nb + 1
        q = swa.swa_qk_norm_rope_append(*(c[n] for n in order), k[:2 * nb], v[:2 * nb], pos + 20, pos,
                                        block_table=table.cuda())
        torch.cuda.synchronize()
        assert torch.equal(q, rows[0])
        assert torch.equal(k, kw) and torch.equal(v, vw)
    record("rotation/valid", lambda: call(None))
    record("rotation/bad page", lambda: call((1, 7)))


if __name__ == "__main__":
    assert swa.swa_version().endswith("debug-checks"), swa.swa_version()
    for kernel in ("simt", "tc", "rows"):
        sinks(kernel)
    rotation()
    swa.swa_set_debug_options()
