"""The decoding loop with attention over the 4-bit cache: graph, eager steps and the definition agree, also over evictions."""
import json
import subprocess
import sys
import os

import numpy as np
import pytest

from oracle import kv4_oracle as K
from oracle.q4_moe_oracle import f64

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def bits(t):
    return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


@pytest.fixture(scope="module")
def make():
    from decode_gemv_sign_gb300 import build
    from decode_gemv_sign_gb300.expert_block import ExpertBlock

    build.build()
    return lambda T, most=128, dim=64: ExpertBlock.random(V=500, H=192, F=80, E=12, top_k=3, group=32, seed=1,
                                                          attention=(6, 2, dim, T, most))


@pytest.mark.parametrize("T", [1, 5])
def test_graph_and_eager_steps_agree(make, T):
    from decode_gemv_sign_gb300 import wcomp

    eager, block = make(T), make(T)
    tokens = torch.arange(T, device="cuda") * 7
    scores = torch.empty(2, T, device="cuda")
    mine = tokens.clone()
    graph = block.graph(mine, *scores)
    assert torch.equal(mine, tokens) and not block.attention.lengths.any() and not block.attention.mass.any()
    for step in range(150):
        if step in (70, 110):
            for b in (eager, block):
                b.attention.evict(40, 10)
            assert (eager.attention.lengths == 40).all()
        tokens, logprob, entropy = eager.scored_step(tokens)
        graph.replay()
        assert torch.equal(mine, tokens) and torch.equal(scores[0], logprob) and torch.equal(scores[1], entropy)
        assert torch.equal(eager.attention.mass, block.attention.mass)
    wcomp.device_check()


def test_a_graph_made_in_the_middle_leaves_the_cache_as_it_was(make):
    """Ten steps, then a graph: its first replay is the eager block's eleventh step; none is made on a full cache."""
    eager, block = make(2), make(2)
    tokens = torch.arange(2, device="cuda") * 5
    for b in (eager, block):
        now = tokens.clone()
        for _ in range(10):
            now = b.scored_step(now)[0]
    mine, scores, mass = now.clone(), torch.empty(2, 2, device="cuda"), block.attention.mass.clone()
    graph = block.graph(mine, *scores)
    assert torch.equal(block.attention.mass, mass) and (block.attention.lengths == 10).all()
    graph.replay()
    want = eager.scored_step(now)
    assert torch.equal(mine, want[0]) and torch.equal(scores[0], want[1]) and torch.equal(scores[1], want[2])
    assert torch.equal(block.attention.mass, eager.attention.mass)
    block.attention.lengths.fill_(block.attention.most)
    with pytest.raises(ValueError):
        block.graph(mine, *scores)


def test_the_attention_is_the_definition(make):
    """Keys, values and queries as the projection gives them; what is gathered decides an eviction."""
    from decode_gemv_sign_gb300 import wcomp

    T = 3
    layer = make(T).attention
    g = torch.Generator(device="cuda").manual_seed(2)
    ks, vs = [[] for _ in range(T)], [[] for _ in range(T)]
    mass = np.zeros((T, 2, layer.most))
    for step in range(90):
        x = torch.randn(T, 192, device="cuda", generator=g).bfloat16()
        y = f64(bits(wcomp.q4_gemv(layer.qkv, x).bfloat16())).reshape(T, 10, 64)
        want = wcomp.q4_gemv(layer.out, layer_out(layer, x).view(T, -1))
        kv = bits(wcomp.q4_gemv(layer.qkv, x).bfloat16()).reshape(T, 10, 64)
        for b in range(T):
            ks[b].append(K.held(kv[b, 6:8]))
            vs[b].append(K.held(kv[b, 8:10]))
            o, _, m, tol, _, mtol = K.attend(y[b:b + 1, :6], np.stack(ks[b]), np.stack(vs[b]), 0.125)
            got = f64(bits(layer.last[b]))
            assert (np.abs(got - o[0]) <= tol[0]).all()
            mass[b, :, :len(ks[b])] += m
        assert torch.isfinite(want).all()
    got = layer.mass.cpu().numpy()
    assert (np.abs(got - mass) <= 1e-4 * mass + 1e-6).all()  # 90 sums of fp32 weights, each off by 2^-19 or so
    before = layer.mass.cpu().numpy()
    layer.evict(30, 8)
    k, _ = wcomp.kv4_read(layer.cache, layer.table, layer.lengths, torch.arange(0, 91, 30, dtype=torch.int32, device="cuda"),
                          rows=90)
    k = f64(bits(k)).reshape(T, 30, 2, 64)
    for b in range(T):
        for h in range(2):
            keep = K.evict(before[b, h], 90, 30, 8)
            assert np.allclose(k[b, :, h], np.stack(ks[b])[keep, h], rtol=2.0 ** -8, atol=0)  # read back in BF16
            assert np.array_equal(layer.mass[b, h, :30].cpu().numpy(), before[b, h, keep])


def layer_out(layer, x):
    """One call of the layer, with what its attention gave kept in layer.last."""
    from decode_gemv_sign_gb300 import wcomp

    inner = wcomp.kv4_attend

    def kept(*a, **k):
        layer.last = inner(*a, **k)
        return layer.last

    wcomp.kv4_attend = kept
    try:
        layer(x)
    finally:
        wcomp.kv4_attend = inner
    return layer.last


@pytest.mark.parametrize("extra", [["--context", "64", "--keep", "16", "--steps", "100"], ["--context", "128", "--steps", "40"]])
def test_the_command(extra):
    r = subprocess.run([sys.executable, "-m", "decode_gemv_sign_gb300.expert_block", "--tokens", "3", "--vocabulary", "512",
                        "--hidden", "256", "--ffn", "128", "--experts", "8", "--top-k", "2", "--heads", "4", "--kv-heads",
                        "2", "--dim", "64", *extra], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    out = json.loads(r.stdout.strip().splitlines()[-1])
    assert out["evictions"] == (1 if "--keep" in extra else 0) and out["mean_entropy"] > 0 > out["mean_logprob"]
    assert len(out["tokens"]) == 3 and out["cache_bytes"] > 0
