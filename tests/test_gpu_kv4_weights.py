"""Weights of cached tokens on both sides of the rules that say how they are found, against their definition."""
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


@pytest.mark.parametrize("D,share", [(64, 1), (64, 8), (64, 9), (64, 10), (64, 11), (64, 16), (64, 17), (128, 8), (128, 9),
                                     (128, 16), (128, 17), (256, 8), (256, 9)])
@pytest.mark.parametrize("window", [0, 700])
def test_weights_by_rows_a_head(W, D, share, window):
    """Tables too wide for a cluster a tile: from kept scores, or from the keys again."""
    b = Batch(W, [2100, 0, 65, 1300], 2, D, seed=share, width=1100)
    q = draw((4, 2 * share, D), np.random.default_rng(D + share), 1.5)
    attend_matches(W, b, q, [1] * 4, starts=False, window=window)
    W.device_check()
