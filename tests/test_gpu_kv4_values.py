"""Attention over cached values from the smallest to the largest that BF16 holds, against the definition in 64 bits.

The softmax does not depend on the values, so neither may the log-sum-exps and the tokens' weights; and what is summed
is at most the largest value, so nothing overflows on the way.
"""
import numpy as np
import pytest

from oracle import kv4_oracle as K
from oracle.q4_moe_oracle import bf16, f64
from test_gpu_kv4 import Batch, attend_matches, bits, dev16, draw, ints

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
@pytest.mark.parametrize("size", [2.0 ** -130, 2.0 ** -120, 1.0, 2.0 ** 90, 2.0 ** 121, 2.0 ** 125])
@pytest.mark.parametrize("way", WAYS)
def test_tokens_far_below_the_largest_score_count(W, D, size, way):
    """One token 5 to 14.8 nats above 4096 others: together they are some of the sum, each alone is little."""
    width, rows = WAYS[way]
    rng = np.random.default_rng(D)
    n = 4097
    k = np.zeros((n, 2, D))
    k[rng.integers(0, n - rows), :, 0] = 14.8
    v = np.clip(rng.standard_normal((n, 2, D)) * size, -2.0 ** 127, 2.0 ** 127)
    b = Batch(W, [n], 2, D, k=bf16(k), v=bf16(v), width=width)
    q = np.zeros((rows, 8, D))
    q[..., 0] = np.linspace(0.33, 1.0, 8)
    attend_matches(W, b, bf16(q), [rows], scale=1.0, starts=way == "rows")
    W.device_check()


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


@pytest.mark.parametrize("D", [64, 128, 256])
def test_small_weights_of_tiny_values(W, D):
    """Products 2^-25.6 of the largest scale's, 2^-120: their sum is the result where the heavy token's value is 0.

    Each is off by at most 2^-11 of itself and 2^-39 of the largest scale, times a code of 7; the result is a BF16 number
    below its normal range, off by half a step of 2^-133 besides.  So many sequences, of the same pages, that a warp has
    all of one.
    """
    n, B, H, s = 2048, 300, 8, 2.0 ** -120
    k, v = np.zeros((n, H, D)), np.full((n, H, D), 7 * s)
    k[0, :, 0], v[0] = 17.72, 0.0
    b = Batch(W, [n], H, D, k=bf16(k), v=bf16(v), width=32)
    q = np.zeros((B, H, D))
    q[..., 0] = 1.0
    out = f64(bits(W.kv4_attend(b.cache, dev16(bf16(q)), b.table.expand(B, 32).contiguous(), b.len.expand(B).contiguous(),
                                scale=1.0)))
    p = 1.0 / (np.exp(b.ks[0][0, 0, 0]) + n - 1)
    want = (n - 1) * p * 7 * s
    tol = (2.0 ** -8 + 2.0 ** -11 + 2.0 ** -20 + n * K.EPS) * want + n * 7 * s * 2.0 ** -39 + 2.0 ** -134
    assert want > 2.0 ** -132 and (np.abs(out - want) <= tol).all(), (out.min(), out.max(), want, tol)
    W.device_check()


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("way", WAYS)
def test_scores_that_are_all_minus_infinity(W, D, way):
    """exp(z - lse) is then NaN, and so are out and the weights; rows that see no token have 0 and add nothing."""
    width, rows = WAYS[way]
    rng = np.random.default_rng(1)
    k = rng.standard_normal((70, 2, D)) / 8
    k[:, :, 3] = -1.0  # a code that is not 0
    b = Batch(W, [70, 0], 2, D, k=bf16(k), width=width)
    q = draw((2 * rows, 8, D), rng)
    q[:, 5, 3] = 0x7F80
    q[:rows, 1, 3] = 0xFF80
    lse, mass = torch.empty(2 * rows, 8, device="cuda"), torch.zeros(2, 2, b.width * 64, device="cuda")
    out = f64(bits(W.kv4_attend(b.cache, dev16(q), b.table, b.len, ints([0, rows, 2 * rows]) if way == "rows" else None,
                                scale=1.0, lse=lse, mass=mass)))
    lse, mass = lse.cpu().numpy(), mass.cpu().numpy()
    assert np.isnan(out[:rows, [1, 5]]).all() and np.isfinite(np.delete(out[:rows], [1, 5], 1)).all()
    assert np.isneginf(lse[:rows, 5]).all() and np.isfinite(np.delete(lse[:rows], [1, 5], 1)).all()
    assert (out[rows:] == 0).all() and np.isneginf(lse[rows:]).all()
    assert np.isnan(mass[0, :, :70 - rows + 1]).all() and (mass[0, :, 70:] == 0).all() and (mass[1] == 0).all()
    W.device_check()
