"""Child process of tests/test_debug_checks_q8_gpu.py: loads the library built with
SWA_DEBUG_CHECKS before anything else does, runs each case over an 8-bit cache and
prints one JSON line per case: {"name", "count" (out-of-range attempts the library
counted), "ok", "detail"}.

Valid inputs count nothing.  Invalid device-side inputs: a sequence length past the
cache and a block-table page outside the pool, which points at pages allocated past
the pool the call is given, so even an unchecked access stays inside memory the test
owns and shows (their rows would dominate any output that read them)."""
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

B, Hq, Hkv, D, L, PAGE, Q, W = 3, 8, 2, 256, 256, 16, 8, 150
N = B * L // PAGE
GUARD = 3
E4M3 = torch.float8_e4m3fn


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def make(page):
    g = torch.Generator(device="cuda").manual_seed(4)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    shape = (N + GUARD, Hkv, PAGE) if page else (B, Hkv, L)
    data = [torch.zeros((*shape, D), dtype=torch.uint8, device="cuda").view(E4M3) for _ in range(2)]
    data += [torch.zeros(shape, dtype=torch.int8, device="cuda") for _ in range(2)]
    table = None
    if page:
        table = torch.arange(N, device="cuda").to(torch.int32).view(B, -1).flip(1).contiguous()
        for t in data[:2]:
            t.view(torch.uint8)[N:] = 0x7e                  # 448
        for t in data[2:]:
            t[N:] = 20
    cache = [t[:N] for t in data] if page else data
    zero = i32([0] * B)
    k, v = rnd(B, L, Hkv, D), rnd(B, L, Hkv, D)
    swa.swa_q8_append(k, v, *cache, zero + L, zero, block_table=table)
    return data, cache, table, rnd(B, Q, Hq, D), rnd(B, Q, Hkv, D)


def record(name, fn):
    torch.cuda.synchronize()
    swa.swa_read_debug_checks()  # clear
    try:
        detail = fn() or ""
        ok = True
    except Exception as e:  # reported to the parent test
        ok, detail = False, repr(e)[:400]
    torch.cuda.synchronize()
    print(json.dumps({"name": name, "count": swa.swa_read_debug_checks(), "ok": ok,
                      "detail": detail}), flush=True)


def equal(a, b):
    assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


lens, pos = i32([256, 200, 90]), i32([248, 192, 82])
for page in (False, True):
    data, cache, table, q, new = make(page)
    tag = "paged" if page else "contiguous"
    bad_table = None
    if page:
        bad_table = table.clone()
        # the last block of sequence 1's positions, and past the rows of its table
        bad_table[1, 192 // PAGE] = N + 1
    for kernel in ("tc", "rows"):
        swa.swa_set_debug_options(force_kernel=kernel)
        call = lambda n, t: swa.swa_q8_verify_attn(q, *cache, n, pos, W, 1 / 16, block_table=t)  # noqa: E731
        want = call(lens, table)
        record(f"attention {kernel} {tag}/valid",
               lambda: [equal(a, b) for a, b in zip(call(lens, table), want)] and "")

        def past():
            got = call(i32([L + 50, 200, 90]), table)
            # (what lies past the cache is not there: sequence 0 sees its 256 rows)
            for a, b in zip(got, want):
                equal(a, b)
        record(f"attention {kernel} {tag}/length past the cache", past)
        if page:
            def outside():
                got = call(lens, bad_table)
                for s in (0, 2):
                    for a, b in zip(got, want):
                        equal(a[s].contiguous(), b[s].contiguous())
                assert got[0].abs().max() < 100
            record(f"attention {kernel} {tag}/page outside the pool", outside)
    swa.swa_set_debug_options()
    rows = swa.swa_q8_read(*cache, lens, pos, Q, block_table=table)
    record(f"read {tag}/valid", lambda: [
        equal(a, b) for a, b in
        zip(swa.swa_q8_read(*cache, lens, pos, Q, block_table=table), rows)] and "")
    record(f"append {tag}/valid", lambda: swa.swa_q8_append(new, new, *cache, lens, pos,
                                                            block_table=table) and "")
    if page:
        rows = swa.swa_q8_read(*cache, lens, pos, Q, block_table=table)

        def read_outside():
            got = swa.swa_q8_read(*cache, lens, pos, Q, block_table=bad_table)
            for s in (0, 2):
                for a, b in zip(got, rows):
                    equal(a[s], b[s])
            assert all(t.isfinite().all() and t.abs().max() < 100 for t in got)
        record("read paged/page outside the pool", read_outside)

        def append_outside():
            before = [t.clone() for t in data]
            swa.swa_q8_append(new * 2, new * 2, *cache, lens, pos, block_table=bad_table)
            torch.cuda.synchronize()
            for a, b in zip(data, before):
                equal(a[N:].contiguous(), b[N:].contiguous())
            got = swa.swa_q8_read(*cache, lens, pos, Q, block_table=table)
            for a, b in zip(got, rows):
                for s in (0, 2):                   # written
                    assert torch.equal(a[s], b[s] * 2)
                assert torch.equal(a[1], b[1])     # dropped
        record("append paged/page outside the pool", append_outside)
