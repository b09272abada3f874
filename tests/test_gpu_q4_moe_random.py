"""Random shapes and forms on three streams at once, against 64 bits on the GPU; each call twice for the same bits."""
import math
import random

import pytest

from oracle import q4_moe_oracle as Q

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def W():
    from decode_gemv_sign_gb300 import build, wcomp

    build.build()
    wcomp.lib()
    return wcomp


@pytest.fixture(scope="module")
def streams():
    return [torch.cuda.Stream() for _ in range(3)]


def log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def values(W, q, K, group):
    codes, scales = W.q4_unpack(q)
    v = torch.stack([codes & 15, codes >> 4], -1).flatten(-2)[..., :K].double() - 8
    return v * scales.double().repeat_interleave(group, -1)[..., :K]


def twice(streams, call):
    """call(i) on each stream, twice: the results of both rounds."""
    torch.cuda.synchronize()
    out = []
    for _ in range(2):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                out.append(call(i))
    torch.cuda.synchronize()
    return out[:3], out[3:]


@pytest.mark.parametrize("seed", range(40))
def test_gemv(W, streams, seed):
    rng = random.Random(seed)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    group, B = rng.choice([32, 64, 128]), rng.randint(1, 16)
    N = log_uniform(rng, 1, 9000)
    K = log_uniform(rng, 1, min(30000, 60_000_000 // N))
    q = W.q4_encode((torch.randn(N, K, device="cuda", generator=g) * 0.02).bfloat16(), group)
    xs = [torch.randn(B, K, device="cuda", generator=g).bfloat16() for _ in streams]
    v = values(W, q, K, group)
    first, second = twice(streams, lambda i: W.q4_gemv(q, xs[i]))
    steps = -(-K // group) + 64
    for x, y, again in zip(xs, first, second):
        assert torch.equal(y, again)
        assert ((y.double() - x.double() @ v.T).abs() <= steps * Q.EPS * (x.double().abs() @ v.abs().T)).all(), (N, K, B, group)
    W.device_check()


@pytest.mark.parametrize("seed", range(40))
def test_moe(W, streams, seed):
    rng = random.Random(1000 + seed)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def bf(*shape, scale=1.0):
        return (torch.randn(*shape, device="cuda", generator=g) * scale).bfloat16()

    E, T, form = log_uniform(rng, 1, 200), rng.randint(1, 16), rng.choice(["bf16", 32, 64, 128])
    k = rng.randint(1, min(E, 16))
    H = log_uniform(rng, 1, 3000)
    F = log_uniform(rng, 1, max(1, min(2000, 40_000_000 // (E * H))))
    if rng.random() < 0.5:  # widths that tensor maps take
        H, F = -(-H // 16) * 16, -(-F // 16) * 16
    scoring, renormalize = rng.choice(["softmax", "sigmoid"]), rng.random() < 0.5
    weights = [bf(E, F, H, scale=H ** -0.5), bf(E, F, H, scale=H ** -0.5), bf(E, H, F, scale=F ** -0.5)]
    if form == "bf16":
        held, (gate, up, down) = weights, [w.double() for w in weights]
    else:
        held = [W.q4_encode(w, form) for w in weights]
        gate, up, down = [values(W, q, K, form) for q, K in zip(held, (H, H, F))]
    router, xs = bf(E, H, scale=2 * H ** -0.5), [bf(T, H) for _ in streams]
    chosen = [(torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda")) for _ in streams]
    first, second = twice(streams, lambda i: W.moe(xs[i], router, *held, k, scoring=scoring, renormalize=renormalize,
                                                   ids=chosen[i][0], weights=chosen[i][1]))
    W.device_check()
    # the bound of oracle.q4_moe_oracle.moe
    lost = Q.TWO_BF16 if form == "bf16" else Q.FP16
    eh, ef = (H / 16 + 64) * Q.EPS, (F * k / 16 + 64) * Q.EPS
    for x, y, again, (ids, p) in zip(xs, first, second, chosen):
        assert torch.equal(y, again)
        assert (torch.sort(ids, 1).values.diff(dim=1) > 0).all() and ((0 <= ids) & (ids < E)).all()
        for t in range(T):
            e, v, xt = ids[t].long(), p[t].double(), x[t].double()
            a, u = gate[e] @ xt, up[e] @ xt
            da, du = eh * (gate[e].abs() @ xt.abs()), eh * (up[e].abs() @ xt.abs())
            silu = a / (1 + torch.exp(-a))
            h = silu * u
            dh = (1.1 * da * (u.abs() + du) + (silu.abs() + 1.1 * da) * du + (lost + 16 * Q.EPS) * h.abs()
                  + 2.0 ** -39 * h.abs().amax(1, keepdim=True))
            want = (v[:, None] * (down[e] @ h[..., None])[..., 0]).sum(0)
            tol = (v[:, None] * (down[e].abs() @ (dh + ef * h.abs())[..., None])[..., 0]).sum(0)
            tol = tol + 2.0 ** -8 * (want.abs() + tol) + 1e-38
            assert ((y[t].double() - want).abs() <= tol).all(), (T, E, k, H, F, form, scoring)
