"""The library built with SWA_DEBUG_CHECKS over an 8-bit cache: runs
tests/debug_checks_q8_run.py in a child process (the binding loads one library per
process).  Valid calls count no out-of-range attempt; a sequence length past the cache
and a page outside the pool are counted, the other sequences are right, and neither a
read nor a store reaches memory past the pool."""
import json
import os
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def results():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sliding_window_speculative_gb300 import build
    build.build(debug_checks=True)
    r = subprocess.run([sys.executable, os.path.join(ROOT, "tests", "debug_checks_q8_run.py")],
                       capture_output=True, text=True, cwd=ROOT, timeout=900)
    lines = [json.loads(x) for x in r.stdout.splitlines() if x.startswith("{")]
    assert r.returncode == 0, r.stderr[-3000:]
    return {x["name"]: x for x in lines}


LAYOUTS = ("contiguous", "paged")
VALID = [f"{c} {t}/valid" for t in LAYOUTS
         for c in ("attention tc", "attention rows", "read", "append")]
INVALID = [f"attention {k} {t}/length past the cache" for t in LAYOUTS for k in ("tc", "rows")] + \
          [f"{c} paged/page outside the pool"
           for c in ("attention tc", "attention rows", "read", "append")]


@pytest.mark.parametrize("name", VALID)
def test_valid_inputs_count_nothing(results, name):
    r = results[name]
    assert r["ok"], r["detail"]
    assert r["count"] == 0, r


@pytest.mark.parametrize("name", INVALID)
def test_out_of_range_inputs_are_counted_and_contained(results, name):
    r = results[name]
    assert r["ok"], r["detail"]
    assert r["count"] > 0, r
