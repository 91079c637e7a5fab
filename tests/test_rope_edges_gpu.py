"""Head norms and rotation with frequencies that are no numbers: NaN in those
pairs, as the definition has it, and nowhere else."""
import numpy as np
import pytest
import torch

import oracle.verify_step as vs
from tests.test_rope_gpu import _case, _f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sliding_window_speculative_gb300 import build
    build.build()
    yield


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,rot", [(64, 64), (128, 64), (256, 256), (256, 16)])
def test_frequencies_that_are_not_finite(D, rot, interleaved):
    import sliding_window_speculative_gb300 as swa
    c = _case(3, 5, 4, 2, D, rot, seed=D + rot, pos=[0, 7, 4000])
    odd = {0: float("nan"), rot // 4: float("inf"), rot // 2 - 1: -float("inf")}
    for n, f in odd.items():
        c["inv_freq"][n] = f
    got = swa.swa_qk_norm_rope(**c, interleaved=interleaved)
    torch.cuda.synchronize()
    pos = (c["q_pos"].cpu().numpy()[:, None] + np.arange(5)).reshape(-1)
    for name, y in zip("qk", got):
        x = _f64(c[name])
        with np.errstate(invalid="ignore"):
            want, size = vs.norm_rope(x.reshape(15, -1, D), _f64(c[name + "_weight"]), c["eps"],
                                      _f64(c["inv_freq"]), pos, interleaved)
        y, bad = _f64(y).reshape(want.shape), np.isnan(want)
        dims = {d for n in odd for d in ((2 * n, 2 * n + 1) if interleaved else (n, n + rot // 2))}
        assert set(np.flatnonzero(bad.any(axis=(0, 1)))) == dims and bad[..., sorted(dims)].all()
        assert np.array_equal(np.isnan(y), bad)
        fine = ~bad
        assert np.all(np.abs(y - want)[fine] <=
                      2.0 ** -8 * np.abs(want)[fine] + 2.0 ** -18 * size[fine])
    assert torch.equal(got[2], c["v"])


def test_a_sound_table_after_a_broken_one():
    import sliding_window_speculative_gb300 as swa
    c = _case(2, 3, 4, 2, 128, 128, seed=9)
    want = [t.clone() for t in swa.swa_qk_norm_rope(**c)]
    f = c["inv_freq"].clone()
    c["inv_freq"].fill_(float("inf"))
    broken = swa.swa_qk_norm_rope(**c)
    assert torch.isnan(broken[0]).all() and torch.isnan(broken[1]).all()
    c["inv_freq"].copy_(f)
    again = swa.swa_qk_norm_rope(**c)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(again, want))
