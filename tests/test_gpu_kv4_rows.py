"""Which positions the rows of a call have: windows up to the largest number."""
import numpy as np
import pytest

from test_gpu_kv4 import Batch, attend_matches, draw

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def W():
    from decode_gemv_sign_gb300 import build, wcomp

    build.build()
    wcomp.lib()
    return wcomp


@pytest.mark.parametrize("D,width", [(64, 7), (128, 7), (256, 7), (64, 1100), (128, 1100), (256, 1100)])
@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 64, 2 ** 31 - 200])
def test_windows_as_large_as_numbers_go(W, D, width, window):
    """They are no window, also for sequences that hold fewer tokens than the call has rows."""
    lengths, rows = [100, 300, 0, 65, 130], [103, 2, 5, 200, 130]
    b = Batch(W, lengths, 2, D, seed=1, width=width)
    q = draw((sum(rows), 4, D), np.random.default_rng(window % 1000), 1.5)
    attend_matches(W, b, q, rows, window=window)
    W.device_check()
