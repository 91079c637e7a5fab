"""The workloads of perf/operators.py: their plain forms, the library's calls
and their 64-bit definitions agree, on the smaller listed cases and on
drawn ones.

Tolerances, as in the operators' own tests but from bounds that need no look
at single keys.  Sinks: a score's summed magnitude is at most
scale |q| |k|, the longest of each (Cauchy-Schwarz); with
d = (D + 8) 2^-24 of it + 2^-20 an output is off by 2^-8 of itself and
(2 d + 2^-14) of the largest |v|, lse by d + 2^-20 + 2^-23 of itself.
Rotation: 2^-8 of the value and 2^-18 (|a| + |b|), where a rotation keeps
a^2 + b^2, so that |a| + |b| is at most twice the row's largest result.
Sampling: whole numbers equal, logprobs within 2^-20 of the value + 2^-34."""
import random

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sliding_window_speculative_gb300 import build
    build.build()
    yield


def _workloads():
    import perf.operators as M
    rng = random.Random(17)
    drawn = [M.draw(rng) for _ in range(60)]
    cases = [c for c in M.listed() if M.work(c)["bytes"] < 1e7]
    cases += [c for c in drawn if M.work(c)["bytes"] < 3e7][:18]
    assert {c["op"] for c in cases} == {"sink", "rope", "sample"} and len(cases) > 18
    return M, cases


def _limits(case, st, i, exact):
    """The bound on |result - exact| of output i."""
    size = exact.abs()
    if case["op"] == "sample":
        return 2.0 ** -20 * size + 2.0 ** -34
    if case["op"] == "rope":
        return 2.0 ** -8 * size + 2.0 ** -17 * size.amax(dim=-1, keepdim=True)
    def longest(t):
        return t.double().square().sum(dim=-1).amax().sqrt()
    d = (case["D"] + 8) * 2.0 ** -24 * case["D"] ** -0.5 * longest(st["q"]) * longest(st["k_cache"])
    d = d + 2.0 ** -20
    if i == 1:
        return d + 2.0 ** -20 + 2.0 ** -23 * size
    return 2.0 ** -8 * size + (2 * d + 2.0 ** -14) * st["v_cache"].double().abs().amax()


def test_plain_forms_calls_and_definitions_agree():
    M, cases = _workloads()
    for n, case in enumerate(cases):
        want = M.exact(dict(case), 100 + n)
        assert want is not None
        for own in (False, True):
            M.own = own
            try:
                st = M.prepare(dict(case), 100 + n)
                got = M.run(st)
                torch.cuda.synchronize()
            finally:
                M.own = False
            for i, (g, w) in enumerate(zip(got, want)):
                if w is None:
                    continue
                what = (case, own, i)
                assert g.shape == w.shape, what
                cache = case["op"] == "sink" and i > 1
                if cache or not g.dtype.is_floating_point or (case["op"] == "rope" and i == 2):
                    # whole numbers, and rows that are copied
                    assert torch.equal(g.double(), w.double()), what
                    continue
                g, w = g.double(), w.double()
                empty = torch.isinf(w)
                assert torch.equal(torch.isinf(g), empty), what
                err = (g - w).abs()
                over = (err > _limits(case, st, i, w)) & ~empty
                assert not over.any(), (what, err[over].max().item())
        del st, got, want
        torch.cuda.empty_cache()
