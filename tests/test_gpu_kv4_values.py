"""Attention over cached values from the smallest to the largest that BF16 holds, against the definition in 64 bits.

The softmax does not depend on the values, so neither may the log-sum-exps and the tokens' weights; and what is summed
is at most the largest value, so nothing overflows on the way.
"""
import numpy as np
import pytest

from oracle.q4_moe_oracle import bf16
from test_gpu_kv4 import Batch, attend_matches, draw

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

# a tile by one cluster; cut anywhere; the same with several rows a sequence
WAYS = {"cluster": (80, 1), "cut": (1100, 1), "rows": (1100, 3)}


@pytest.fixture(scope="module")
def W():
    from decode_gemv_sign_gb300 import build, wcomp

    build.build()
    wcomp.lib()
    return wcomp


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("way", WAYS)
@pytest.mark.parametrize("n", [300, 4097])
def test_many_tokens_of_the_largest_values(W, D, way, n):
    """Weights alike: the result is the values' mean, though their sum is beyond fp32."""
    width, rows = WAYS[way]
    rng = np.random.default_rng(n)
    v = 2.0 ** 127 * (1 - rng.random((n, 2, D)) / 8)
    v[:, 1] *= rng.choice([-1.0, 1.0], (n, D))
    b = Batch(W, [n], 2, D, k=bf16(rng.standard_normal((n, 2, D)) / 8), v=bf16(v), width=width)
    on, _, _ = attend_matches(W, b, draw((rows, 8, D), rng), [rows], starts=way == "rows")
    assert np.isfinite(on).all()
    W.device_check()
