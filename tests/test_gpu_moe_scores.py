"""Scores far below one: the choice goes by them as long as fp32 tells them apart."""
import numpy as np
import pytest

from test_gpu_moe import Layer, check, dev

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def W():
    from decode_gemv_sign_gb300 import build, wcomp

    build.build()
    wcomp.lib()
    return wcomp


def with_logits(layer, logits):
    """Every token's logit of expert e is logits[e] (BF16 values)."""
    layer.x[:] = 0
    layer.x[:, 0] = 0x3F80
    layer.router[:] = 0
    layer.router[:, 0] = (np.asarray(logits, np.float32).view(np.uint32) >> 16).astype(np.uint16)


@pytest.mark.parametrize("E", [12, 150, 300, 1024])
def test_small_sigmoid_scores_are_told_apart(W, E):
    """Logits of -89 to -100 have scores of 2^-128 to 2^-144: the largest are chosen, not the lowest indexes."""
    layer = Layer(W, 2, E, 64, 8, "bf16", seed=E)
    logits = np.full(E, -200.0)
    at = np.arange(12) * (E // 12)
    logits[at] = -100.0 + np.arange(12)
    with_logits(layer, logits)
    ids = torch.full((2, 6), -1, dtype=torch.int32, device="cuda")
    weights = torch.zeros(2, 6, device="cuda")
    W.moe(dev(layer.x), dev(layer.router), *layer.dev, 6, scoring="sigmoid", renormalize=False, ids=ids, weights=weights)
    assert (ids.cpu().numpy() == at[:5:-1]).all()
    want = np.exp(logits[at[:5:-1]])
    # two steps of the smallest fp32 value, and of the exponential's last bit
    assert (np.abs(weights.cpu().numpy() - want) <= 2.0 ** -148 + 2.0 ** -21 * want).all()


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E", [20, 200, 400])
def test_scores_over_the_whole_range(W, E, scoring):
    """Logits from -120 to 120, and 88 where exp nearly overflows, either sign."""
    layer = Layer(W, 3, E, 64, 8, "bf16", seed=E)
    logits = np.linspace(-120.0, 120.0, E).round()
    logits[[0, 3, 5, 7]] = [88.5, -88.5, 87.5, -87.5]
    with_logits(layer, logits)
    check(W, layer, 5, scoring, renormalize=False)


def test_infinite_logits(W):
    """Sigmoid scores of +-inf are 1 and 0."""
    layer = Layer(W, 1, 5, 32, 8, "bf16", seed=3)
    with_logits(layer, [-np.inf, 0.0, np.inf, -1.0, 1.0])
    ids, weights = torch.zeros(1, 5, dtype=torch.int32, device="cuda"), torch.zeros(1, 5, device="cuda")
    W.moe(dev(layer.x), dev(layer.router), *layer.dev, 5, scoring="sigmoid", renormalize=False, ids=ids, weights=weights)
    assert ids.tolist() == [[2, 4, 1, 3, 0]]
    assert weights[0, 0] == 1 and weights[0, 2] == 0.5 and weights[0, 4] == 0
