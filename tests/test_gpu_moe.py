"""The mixture-of-experts layer against its definition in 64 bits.

The choice is checked by the scores (every chosen expert is within the scores'
fp32 error of the k best), the weights against the scores, and y for that
choice against the error bound derived in oracle.q4_moe_oracle.moe.
"""
import numpy as np
import pytest

from decode_gemv_sign_gb300 import synth
from oracle import q4_moe_oracle as Q

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def W():
    from decode_gemv_sign_gb300 import build, wcomp

    build.build()
    wcomp.lib()
    return wcomp


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a).view(np.int16)).cuda().view(torch.bfloat16)


def bits(t):
    return t.view(torch.int16).cpu().numpy().view(np.uint16)


class Layer:
    def __init__(self, W, T, E, H, F, form, seed):
        rng = np.random.default_rng(seed)

        def draw(shape, sigma):
            return Q.bf16(rng.standard_normal(shape) * sigma)

        self.held = Q.TWO_BF16 if form == "bf16" else Q.FP16
        self.x = draw((T, H), 1.0)
        self.router = draw((E, H), 2.0 / np.sqrt(H))
        ws = [draw((E, F, H), 1.0 / np.sqrt(H)), draw((E, F, H), 1.0 / np.sqrt(H)), draw((E, H, F), 1.0 / np.sqrt(F))]
        if form == "bf16":
            self.dev = [dev(w) for w in ws]
            self.values = [Q.f64(w) for w in ws]
        else:
            self.dev = [W.q4_encode(dev(w), form) for w in ws]
            self.values = [Q.q4_values(*Q.q4_encode(w, form), form) for w in ws]


def check(W, layer, k, scoring="softmax", bias=None, renormalize=True, factor=1.0, x=None):
    x = layer.x if x is None else x
    T, E = x.shape[0], layer.router.shape[0]
    ids = torch.full((T, k), -1, dtype=torch.int32, device="cuda")
    weights = torch.full((T, k), float("nan"), device="cuda")
    xd = dev(x)
    kw = dict(scoring=scoring, renormalize=renormalize, factor=factor,
              bias=None if bias is None else torch.from_numpy(bias).cuda())
    y = W.moe(xd, dev(layer.router), *layer.dev, k, ids=ids, weights=weights, **kw)
    W.device_check()
    assert y.dtype == torch.bfloat16 and y.shape == xd.shape
    ids, weights = ids.cpu().numpy(), weights.cpu().numpy().astype(np.float64)
    # the choice
    s, ds = Q.scores(x, layer.router, scoring)
    by = s if bias is None else s + bias.astype(np.float64)
    eb = ds + (0 if bias is None else Q.EPS * (np.abs(by) + 1e-30))
    assert ((0 <= ids) & (ids < E)).all()
    rows = np.arange(T)[:, None]
    assert (np.sort(ids, 1)[:, 1:] != np.sort(ids, 1)[:, :-1]).all()
    best = np.sort(by, 1)[:, ::-1][:, :k]
    for j in range(k):
        got = by[rows[:, 0], ids[:, j]]
        slack = 2 * eb.max(1)
        ok = (got >= best[:, j] - slack) & (got <= best[:, j] + slack) | (got == best[:, j])
        assert ok.all()
    # the weights
    p = s[rows, ids]
    if renormalize:
        want = factor * p / np.maximum(p.sum(1, keepdims=True), 1e-20)
        dw = np.abs(want) * (2 * (ds[rows, ids] / p).max(1, keepdims=True) + 32 * Q.EPS)
    else:
        want, dw = factor * p, abs(factor) * (ds[rows, ids] + 4 * Q.EPS * p)
    assert (np.abs(weights - want) <= dw).all()
    # the layer's output for that choice and those weights
    want, tol = Q.moe(x, *layer.values, ids, weights, layer.held)
    assert (np.abs(Q.f64(bits(y)) - want) <= tol).all()
    # the same bits again
    assert torch.equal(W.moe(xd, dev(layer.router), *layer.dev, k, **kw).view(torch.int16), y.view(torch.int16))
    return ids, weights, y


@pytest.mark.parametrize("form", ["bf16", 32, 64, 128])
@pytest.mark.parametrize("T,E,k,H,F", [
    (1, 1, 1, 1, 1), (1, 4, 2, 64, 32), (3, 5, 5, 17, 9), (16, 1, 1, 257, 129), (16, 2, 1, 128, 128),
    (2, 130, 16, 96, 40), (16, 8, 2, 256, 512), (5, 12, 3, 1001, 333), (9, 7, 4, 520, 264), (1, 64, 8, 1024, 256)])
def test_layer(W, T, E, k, H, F, form):
    check(W, Layer(W, T, E, H, F, form, seed=T + E + H), k)


@pytest.mark.parametrize("T,E,k", [(16, 129, 3), (3, 256, 16), (7, 257, 8), (2, 300, 1), (16, 1024, 16)])
def test_many_experts(W, T, E, k):
    check(W, Layer(W, T, E, 72, 8, "bf16", seed=E), k)
    rng = np.random.default_rng(E)
    layer = Layer(W, T, E, 64, 8, 32, seed=E + 1)
    check(W, layer, k, "sigmoid", rng.standard_normal(E).astype(np.float32))


@pytest.mark.parametrize("form", ["bf16", 32, 128])
@pytest.mark.parametrize("T,E,k,H,F", [(1, 2, 1, 8192, 40), (1, 2, 1, 40, 8200), (16, 2, 2, 4100, 32), (9, 3, 2, 33, 5001),
                                       (16, 3, 3, 2048, 70)])
def test_few_long_rows(W, T, E, k, H, F, form):
    """Fewer tiles than thread blocks: their sums are cut along the rows and joined."""
    check(W, Layer(W, T, E, H, F, form, seed=H + F), k)


@pytest.mark.parametrize("H,F", [(64, 64), (40, 72), (1001, 333), (33, 35)])
def test_what_is_not_chosen_is_not_read_into_the_sums(W, H, F):
    """Experts that no token chose, and the rows next to a tile's edge, may hold anything."""
    layer = Layer(W, 10, 5, H, F, "bf16", seed=H)
    bias = np.array([0, -np.inf, 0, -np.inf, 0], np.float32)
    for w in layer.dev:
        w[1] = float("nan")
        w[3] = float("inf")
    check(W, layer, 3, "sigmoid", bias)
    # one row of `down`: one column of y
    row = H // 2
    layer.dev[2][:, row] = float("nan")
    y = W.moe(dev(layer.x), dev(layer.router), *layer.dev, 3, scoring="sigmoid", bias=torch.from_numpy(bias).cuda())
    bad = torch.isnan(y)
    assert bad[:, row].all() and bad.sum() == 10


@pytest.mark.parametrize("form", ["bf16", 64])
def test_infinite_hidden_values_keep_their_sign(W, form):
    """A gate and an up row of large weights overflow one hidden value: y is what 64 bits call infinite."""
    layer = Layer(W, 1, 1, 64, 64, "bf16", seed=2)
    layer.x[:] = 0x3F80
    w = [Q.bf16(np.clip(v, -0.5, 0.5)) for v in layer.values]
    w[0][0, 5] = w[1][0, 5] = 0x7E00  # 64 of them: 2.7e39
    w[2][:] = Q.bf16(np.where(np.arange(64) % 2, 0.5, -0.5))[None, :, None]
    weights = [dev(a) if form == "bf16" else W.q4_encode(dev(a), form) for a in w]
    y = W.moe(dev(layer.x), dev(layer.router), *weights, 1).float().cpu().numpy()[0]
    assert (y == np.where(np.arange(64) % 2, np.inf, -np.inf)).all()


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [False, True])
@pytest.mark.parametrize("biased", [False, True])
def test_routing_variants(W, scoring, renormalize, biased):
    layer = Layer(W, 11, 40, 320, 48, "bf16", seed=5)
    bias = np.random.default_rng(2).standard_normal(40).astype(np.float32) * 0.3 if biased else None
    check(W, layer, 6, scoring, bias, renormalize, factor=2.5)


def test_all_tokens_on_one_expert_and_all_on_different_ones(W):
    layer = Layer(W, 16, 16, 128, 64, "bf16", seed=8)
    bias = np.zeros(16, np.float32)
    bias[5] = 10.0
    ids, _, _ = check(W, layer, 1, "sigmoid", bias)
    assert (ids == 5).all()
    x = np.zeros((16, 128), np.uint16)
    x[np.arange(16), np.arange(16)] = 0x4120  # 10
    layer.router = np.zeros((16, 128), np.uint16)
    layer.router[np.arange(16), np.arange(16)] = 0x3F80
    ids, _, _ = check(W, layer, 1, x=x)
    assert (ids[:, 0] == np.arange(16)).all()


def test_ties_go_to_the_lowest_index(W):
    layer = Layer(W, 3, 50, 64, 32, "bf16", seed=3)
    layer.router[:] = 0  # every score the same
    ids, weights, _ = check(W, layer, 4)
    assert (ids == np.arange(4)).all()
    assert np.allclose(weights, 0.25, rtol=1e-6)


@pytest.mark.parametrize("low", [-np.inf, np.finfo(np.float32).min])
def test_masked_experts(W, low):
    """A bias of -inf, or of the type's lowest value, keeps an expert out while others are left."""
    layer = Layer(W, 6, 20, 64, 32, "bf16", seed=4)
    bias = np.full(20, low, np.float32)
    open_ = [3, 7, 8, 19]
    bias[open_] = 0
    for k in (1, 4):
        ids, _, _ = check(W, layer, k, "sigmoid", bias)
        assert np.isin(ids, open_).all()
    # more wanted than open: the masked ones of lowest index follow
    ids = torch.zeros(6, 6, dtype=torch.int32, device="cuda")
    W.moe(dev(layer.x), dev(layer.router), *layer.dev, 6, bias=torch.from_numpy(bias).cuda(), ids=ids)
    got = ids.cpu().numpy()
    assert (np.sort(got[:, :4], 1) == open_).all()
    assert (got[:, 4:] == [0, 1]).all()


def test_nan_token_stays_alone(W):
    layer = Layer(W, 7, 24, 160, 64, "bf16", seed=6)
    _, _, clean = check(W, layer, 3)
    x = layer.x.copy()
    x[2, 100] = 0x7FC0
    ids = torch.full((7, 3), -1, dtype=torch.int32, device="cuda")
    y = W.moe(dev(x), dev(layer.router), *layer.dev, 3, ids=ids)
    W.device_check()
    assert torch.isnan(y[2]).all()
    keep = [t for t in range(7) if t != 2]
    # other experts are at work, so sums may be cut elsewhere: a BF16 step of the largest value
    assert (y[keep].float() - clean[keep].float()).abs().max() <= 2.0 ** -7 * clean[keep].float().abs().max()
    assert (ids[2].cpu().numpy() == [0, 1, 2]).all()  # a NaN ranks below everything: the lowest indexes are left


def test_infinite_router_logit(W):
    """One expert's logit of -inf gives it score 0."""
    layer = Layer(W, 2, 6, 32, 32, "bf16", seed=7)
    layer.x[:, 0] = 0x3F80
    layer.router[4, 0] = 0xFF80
    ids = torch.zeros(2, 5, dtype=torch.int32, device="cuda")
    y = W.moe(dev(layer.x), dev(layer.router), *layer.dev, 5, ids=ids)
    assert not (ids == 4).any() and torch.isfinite(y).all()


def test_negative_and_large_gates(W):
    """silu at its ends: gates far below zero give 0, far above give the gate itself."""
    layer = Layer(W, 4, 2, 64, 32, "bf16", seed=10)
    layer.values[0] = layer.values[0] * 256.0
    layer.dev[0] = dev(Q.bf16(layer.values[0]))
    check(W, layer, 2)


@pytest.mark.parametrize("off", [1, 8])
@pytest.mark.parametrize("form", ["bf16", 64])
def test_unaligned_inputs(W, off, form):
    layer = Layer(W, 3, 6, 64, 48, form, seed=12)
    want = W.moe(dev(layer.x), dev(layer.router), *layer.dev, 2)

    def moved(t):
        buf = torch.zeros(t.numel() + off, dtype=t.dtype, device="cuda")
        buf[off:].copy_(t.reshape(-1))
        return buf[off:].view(t.shape)

    ws = [moved(w) for w in layer.dev] if form == "bf16" else layer.dev
    got = W.moe(moved(dev(layer.x)), moved(dev(layer.router)), *ws, 2)
    # other paths may add in another order: both within the layer's own bound, here a BF16 step
    assert (got.float() - want.float()).abs().max() <= 2.0 ** -7 * want.float().abs().max()
    assert torch.equal(W.moe(moved(dev(layer.x)), dev(layer.router), *layer.dev, 2), want)


def test_y_may_be_x(W):
    layer = Layer(W, 8, 10, 256, 64, "bf16", seed=13)
    want = W.moe(dev(layer.x), dev(layer.router), *layer.dev, 2)
    x = dev(layer.x)
    W.moe(x, dev(layer.router), *layer.dev, 2, y=x)
    assert torch.equal(x, want)
    # bits in, bits out
    assert torch.equal(W.moe(dev(layer.x).view(torch.int16), dev(layer.router), *layer.dev, 2), want.view(torch.int16))


def test_offsets_past_32_bits(W):
    """Experts that start more than 2^32 elements into the stack."""
    E, H, F = 70, 8192, 8192
    w = torch.zeros(E, F, H, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    last = [torch.empty(F, H, dtype=torch.bfloat16, device="cuda").normal_(0, 0.01, generator=g) for _ in range(1)][0]
    w[E - 1] = last
    assert (E - 1) * F * H > 2 ** 32
    x = torch.empty(1, H, dtype=torch.bfloat16, device="cuda").normal_(0, 1, generator=g)
    router = torch.zeros(E, H, dtype=torch.bfloat16, device="cuda")
    bias = torch.zeros(E, device="cuda")
    bias[E - 1] = 1.0
    y = W.moe(x, router, w, w, w, 1, bias=bias)
    h = last.double() @ x[0].double()
    h = h / (1 + torch.exp(-h)) * h
    want = last.double() @ h
    err = (y[0].double() - want).abs()
    # one BF16 rounding, and 16 bits of every hidden value
    assert (err <= 2.0 ** -8 * want.abs() + 2.0 ** -16 * (last.double().abs() @ h.abs())).all()
    del w


def test_two_streams(W):
    layers = [Layer(W, 4, 16, 512, 256, "bf16", seed=20 + i) for i in range(2)]
    args = [(dev(a.x), dev(a.router), *a.dev, 4) for a in layers]
    want = [W.moe(*a) for a in args]
    streams = [torch.cuda.Stream() for _ in args]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(W.moe(*args[i]))
    torch.cuda.synchronize()
    W.device_check()
    for i in range(2):
        assert all(torch.equal(y, want[i]) for y in got[i])


def test_in_a_graph(W):
    layer = Layer(W, 2, 16, 512, 256, "bf16", seed=30)
    x, router = dev(layer.x), dev(layer.router)
    y = torch.zeros_like(x)
    W.moe(x, router, *layer.dev, 4, y=y)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        W.moe(x, router, *layer.dev, 4, y=y)
    x.copy_(x.flip(0))
    for _ in range(3):
        y.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, W.moe(x, router, *layer.dev, 4))
    W.device_check()


def test_a_graph_next_to_many_calls(W):
    """A captured call has counters of its own, whatever runs next to it."""
    layer = Layer(W, 2, 16, 512, 256, 64, seed=31)
    x, router = dev(layer.x), dev(layer.router)
    want = W.moe(x, router, *layer.dev, 4)
    # rows shared by clusters, and rows cut and joined in memory
    cs = [W.q4_encode(torch.randn(*shape, device="cuda").bfloat16(), 64) for shape in ((64, 40000), (9744, 14350))]
    vs = [torch.randn(12, 40000, device="cuda").bfloat16(), torch.randn(1, 14350, device="cuda").bfloat16()]
    products = [W.q4_gemv(c, v) for c, v in zip(cs, vs)]
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        y, zs = torch.zeros_like(x), [torch.zeros_like(p) for p in products]
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            for _ in range(10):
                W.moe(x, router, *layer.dev, 4, y=y)
                for c, v, z in zip(cs, vs, zs):
                    W.q4_gemv(c, v, z)
        graphs.append((g, [y, *zs], torch.cuda.Stream()))
    torch.cuda.synchronize()
    out = []
    for i in range(120):
        for g, held, s in graphs:
            with torch.cuda.stream(s):
                if i % 4 == 0:
                    for t in held:
                        t.zero_()
                g.replay()
        out.append([W.moe(x, router, *layer.dev, 4) for _ in range(10)][-1:] + [W.q4_gemv(c, v) for c, v in zip(cs, vs)])
    torch.cuda.synchronize()
    W.device_check()
    for held in (*out, *(held for _, held, _ in graphs)):
        assert all(torch.equal(a, b) for a, b in zip(held, [want, *products]))


def test_more_captured_calls_than_kept_counters(W):
    layer = Layer(W, 1, 2, 8, 8, 32, seed=32)
    x, router = dev(layer.x), dev(layer.router)
    want = W.moe(x, router, *layer.dev, 1)
    torch.cuda.synchronize()
    for _ in range(11):
        y = torch.zeros_like(x)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            for _ in range(400):
                W.moe(x, router, *layer.dev, 1, y=y)
        g.replay()
        assert torch.equal(y, want)
        del g
    W.device_check()


def test_refusals(W):
    T, E, H, F = 2, 6, 64, 32
    x = torch.zeros(T, H, dtype=torch.bfloat16, device="cuda")
    r = torch.zeros(E, H, dtype=torch.bfloat16, device="cuda")
    gu = torch.zeros(E, F, H, dtype=torch.bfloat16, device="cuda")
    d = torch.zeros(E, H, F, dtype=torch.bfloat16, device="cuda")
    W.moe(x, r, gu, gu, d, 2)
    for k in (0, 7):
        with pytest.raises(W.WcompError):
            W.moe(x, r, gu, gu, d, k)
    with pytest.raises(W.WcompError):
        W.moe(torch.zeros(17, H, dtype=torch.bfloat16, device="cuda"), r, gu, gu, d, 2)
    with pytest.raises(W.WcompError):
        W.moe(x[:0], r, gu, gu, d, 2)
    for bad in ((x[0], r, gu, gu, d), (x, r[:, :32].contiguous(), gu, gu, d), (x, r[:5], gu, gu, d),
                (x, r, gu, gu[:, :16].contiguous(), d), (x, r, gu, gu, gu), (x, r, gu[0], gu, d)):
        with pytest.raises(ValueError):
            W.moe(*bad, 2)
    with pytest.raises(TypeError):
        W.moe(x.float(), r, gu, gu, d, 2)
    with pytest.raises(TypeError):
        W.moe(x, r.cpu(), gu, gu, d, 2)
    q = W.q4_encode(gu, 32)
    with pytest.raises(TypeError):
        W.moe(x, r, q, gu, d, 2)
    with pytest.raises(W.WcompError):  # one group size for all three
        W.moe(x, r, q, q, W.q4_encode(d, 64), 2)
    with pytest.raises(ValueError):
        W.moe(x, r, gu, gu, d, 2, scoring="relu")
    with pytest.raises(ValueError):
        W.moe(x, r, gu, gu, d, 2, bias=torch.zeros(E + 1, device="cuda"))
    with pytest.raises(ValueError):
        W.moe(x, r, gu, gu, d, 2, ids=torch.zeros(T, 2, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        W.moe(x, r, gu, gu, d, 2, y=x[:1])
    big = torch.zeros(1025, 8, dtype=torch.bfloat16, device="cuda")
    w = torch.zeros(1025, 8, 8, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(W.WcompError):
        W.moe(torch.zeros(1, 8, dtype=torch.bfloat16, device="cuda"), big, w, w, w, 2)
    with pytest.raises(W.WcompError):
        W.moe(torch.zeros(1, 8, dtype=torch.bfloat16, device="cuda"), big[:100], w[:100], w[:100], w[:100], 17)
