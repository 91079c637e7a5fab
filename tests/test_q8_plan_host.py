"""The workspace bound of the attention over the 8-bit cache where a plan has more splits
than were asked for (no chunk exceeds 8192 keys), or none at all."""
import pytest

import sliding_window_speculative_gb300 as swa
from sliding_window_speculative_gb300 import build


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


def partials(dims, splits):
    return dims.batch * dims.q_len * dims.num_q_heads * splits * (dims.head_dim + 2) * 4


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("asked,window,splits", [
    (1, 8185, 1), (1, 8186, 2), (1, 40000, 5), (3, 40000, 5), (7, 40000, 7), (0, 40000, 64),
    (1, 64 * 8192 - 7, 64)])
def test_forced_splits(D, asked, window, splits):
    dims = swa.make_dims(2, 8, 8, 2, D, 1 << 20, asked)
    need = swa.swa_q8_workspace_bytes(dims, window)
    # (one split needs no partials)
    assert need == (partials(dims, splits) if splits > 1 or asked == 0 else 0)


def test_windows_past_the_splits():
    """More than 64 chunks: the windows' bf16 rows."""
    dims = swa.make_dims(2, 8, 8, 2, 128, 1 << 20, 1)
    assert swa.swa_q8_workspace_bytes(dims, 64 * 8192) >= 2 * 2 * 2 * (64 * 8192) * 128 * 2


def test_rows_of_narrow_windows_keep_one_split():
    """A long block whose rows each see few keys asks for no more splits."""
    dims = swa.make_dims(2, 512, 8, 2, 64, 1 << 20, 1)
    assert swa.swa_q8_workspace_bytes(dims, 8000) == 0
    assert swa.swa_q8_workspace_bytes(dims, 8192) == partials(dims, 2)
