"""4-bit products whose scales and activations have far apart exponents.

Only the product of a scale and an activation has to be in range: a scale of
2^110 with activations of 2^-110 gives ordinary results, and so do hidden values
near fp32's largest with small scales of the down projection.
"""
import numpy as np
import pytest

from oracle import q4_moe_oracle as Q
from test_gpu_moe import Layer, check
from test_gpu_q4 import dev

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def W():
    from decode_gemv_sign_gb300 import build, wcomp

    build.build()
    wcomp.lib()
    return wcomp


def held(W, codes, scales, K, group):
    return W.q4_pack(torch.from_numpy(Q.pack_codes(codes)).cuda(), dev(scales).view(torch.bfloat16), K, group)


@pytest.mark.parametrize("group", [32, 64, 128])
def test_one_group_by_hand(W, group):
    """Codes 15, scale 2^110, x = 2^-100, 32 columns: 7 * 32 * 2^10."""
    K = 32
    codes, scales = np.full((1, K), 15, np.uint8), Q.bf16(np.full((1, 1), 2.0 ** 110))
    x = Q.bf16(np.full((1, K), 2.0 ** -100))
    y = W.q4_gemv(held(W, codes, scales, K, group), dev(x))
    assert y.item() == 7 * 32 * 2.0 ** 10


@pytest.mark.parametrize("B", [1, 8, 16])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("N,K", [(70, 1100), (40, 40000)])
def test_gemv_with_scales_against_x(W, N, K, group, B):
    """Scales from 2^-110 to 2^110, another exponent for each 128 columns, against x of the opposite exponent."""
    rng = np.random.default_rng(N + group + B)
    p = np.concatenate([[-110.0, 110.0], rng.integers(-110, 111, -(-K // 128))])[:-(-K // 128)]
    groups = -(-K // group)
    codes = rng.integers(0, 16, (N, K)).astype(np.uint8)
    scales = Q.bf16(rng.uniform(0.5, 2.0, (N, groups)) * 2.0 ** p[np.arange(groups) * group // 128])
    x = Q.bf16(rng.standard_normal((B, K)) * 2.0 ** -p[np.arange(K) // 128])
    v = Q.q4_values(codes, scales, group)
    want, tol = Q.gemv(v, x, group)
    xv = np.abs(Q.f64(x))
    for k in range(0, K, 128):  # what x itself may lose
        tol = tol + 2.0 ** -39 * xv[:, k:k + 128].max(1, keepdims=True) * np.abs(v[:, k:k + 128]).sum(1)
    y = W.q4_gemv(held(W, codes, scales, K, group), dev(x)).cpu().numpy()
    assert (np.abs(y - want) <= tol).all()
    W.device_check()


@pytest.mark.parametrize("T,E,k,H,F", [(1, 4, 2, 256, 160), (5, 3, 2, 200, 300), (16, 1, 1, 128, 256), (11, 2, 2, 130, 70)])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_experts_with_scales_against_their_inputs(W, T, E, k, H, F, group):
    """x of 2^-116 with gate and up weights of 2^116, then hidden values of 2^124 with down weights of 2^-110."""
    layer = Layer(W, T, E, H, F, "bf16", seed=T + group)
    layer.held = Q.FP16
    layer.x = Q.bf16(Q.f64(layer.x) * 2.0 ** -116)
    layer.router = Q.bf16(Q.f64(layer.router) * 2.0 ** 116)
    gate, up, down = layer.values
    experts = [Q.bf16(w * 2.0 ** e) for w, e in ((gate, 116), (up, 116), (down, 0))]
    wide = [Q.bf16(w * 2.0 ** e) for w, e in ((gate, 0), (up, 124), (down, -110))]
    for ws, x, router in ((experts, layer.x, layer.router),
                          (wide, Q.bf16(Q.f64(layer.x) * 2.0 ** 116), Q.bf16(Q.f64(layer.router) * 2.0 ** -116))):
        layer.x, layer.router = x, router
        layer.dev = [W.q4_encode(dev(w), group) for w in ws]
        layer.values = [Q.q4_values(*Q.q4_encode(w, group), group) for w in ws]
        check(W, layer, k)
