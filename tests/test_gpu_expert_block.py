"""The decoding loop over a quantised block: the captured step, the eager one and the definition agree."""
import numpy as np
import pytest

from oracle import q4_moe_oracle as Q

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def bits(t):
    return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


@pytest.fixture(scope="module")
def block():
    from decode_gemv_sign_gb300 import build
    from decode_gemv_sign_gb300.expert_block import ExpertBlock

    build.build()
    return ExpertBlock.random(V=500, H=192, F=80, E=12, top_k=3, group=32, seed=1)


@pytest.mark.parametrize("T", [1, 4, 16])
def test_graph_and_eager_steps_agree(block, T):
    from decode_gemv_sign_gb300 import wcomp

    start = torch.arange(T, device="cuda") * 7
    eager = [start]
    for _ in range(5):
        eager.append(block.step(eager[-1]))
    tokens = start.clone()
    graph = block.graph(tokens)
    for want in eager[1:]:
        graph.replay()
        assert torch.equal(tokens, want)
    wcomp.device_check()


def test_hidden_is_the_definition(block):
    """Within the layer's bound plus two BF16 roundings of the residual stream (2^-8 each) and what they move."""
    from decode_gemv_sign_gb300 import wcomp

    x = block.embed[torch.arange(6, device="cuda")]
    values = []
    for c in (block.proj, *block.experts):
        codes, scales = wcomp.q4_unpack(c)
        codes = codes.cpu().numpy()
        codes = np.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], -1)
        values.append(Q.q4_values(codes, bits(scales), 32))
    r64 = Q.f64(bits(x)) + Q.f64(bits(x)) @ values[0].T
    r = (x.float() + wcomp.q4_gemv(block.proj, x)).bfloat16()
    assert (np.abs(Q.f64(bits(r)) - r64) <= 2.0 ** -8 * np.abs(r64) + 1e-4).all()
    ids = torch.zeros(6, 3, dtype=torch.int32, device="cuda")
    weights = torch.zeros(6, 3, device="cuda")
    wcomp.moe(r, block.router, *block.experts, 3, ids=ids, weights=weights)
    y, tol = Q.moe(bits(r), *values[1:], ids.cpu().numpy(), weights.cpu().numpy().astype(np.float64), Q.FP16)
    want = Q.f64(bits(r)) + y
    assert (np.abs(Q.f64(bits(block.hidden(x))) - want) <= tol + 2.0 ** -8 * (np.abs(want) + tol)).all()
