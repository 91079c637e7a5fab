"""Token log probabilities at the borders of the rule that gives a row one, two, four or
eight CTAs and a CTA its threads: rows and columns on either side, against the fp64
definition within the bounds of tests/test_logprobs_gpu.py."""
import numpy as np
import pytest
import torch

from tests.test_logprobs_gpu import check, logits

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sliding_window_speculative_gb300 import build
    build.build()
    yield


@pytest.mark.parametrize("V,rows", [
    (16370, 57), (16390, 57), (32760, 76), (32800, 76), (65500, 28), (65540, 28), (65540, 29),
    (66000, 40), (66000, 57), (100352, 1), (100352, 28), (131071, 20), (140000, 57), (262100, 9),
    (262144, 9), (262144, 10), (262144, 20), (262144, 28), (262144, 29), (262144, 58)])
@pytest.mark.parametrize("top", [0, 20])
def test_rows_shared_by_clusters(V, rows, top):
    x = logits(1, rows, V, seed=V + rows)
    tok = np.random.default_rng(rows).integers(0, V, (1, rows))
    tok[0, 0] = int(x[0, 0].float().argmax())
    check(x, tok, top, T=[0.8], rows=[(0, 0), (0, rows // 2), (0, rows - 1)])
