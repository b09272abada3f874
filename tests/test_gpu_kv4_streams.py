"""The cache's calls next to one another: on streams, in graphs, in graphs next to eager calls; and at offsets past 2^32."""
import numpy as np
import pytest

from oracle import kv4_oracle as K
from oracle.q4_moe_oracle import f64
from test_gpu_kv4 import Batch, attend_matches, bits, dev16, draw, ints, same_values, starts_of

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def W():
    from decode_gemv_sign_gb300 import build, wcomp

    build.build()
    wcomp.lib()
    return wcomp


# one cluster a tile; cut anywhere; several rows a sequence; dims of each kernel
SHAPES = [([700], 2, 128, 4, [1]), ([3000, 20, 0, 900], 2, 128, 4, [1] * 4), ([2000, 90], 3, 64, 5, [4, 3]),
          ([500] * 40, 4, 64, 1, [1] * 40), ([1500, 64], 1, 256, 9, [1, 2])]


def calls(W, seed):
    out = []
    for i, (lengths, H, D, share, rows) in enumerate(SHAPES):
        b = Batch(W, lengths, H, D, seed=seed + i)
        q = dev16(draw((sum(rows), H * share, D), np.random.default_rng(seed + i), 1.5))
        starts = starts_of(rows)

        def call(b=b, q=q, starts=starts):
            lse = torch.empty(q.shape[:2], device="cuda")
            mass = torch.zeros(len(b.lengths), b.H, b.width * 64, device="cuda")
            return W.kv4_attend(b.cache, q, b.table, b.len, starts, lse=lse, mass=mass), lse, mass

        out.append(call)
    return out


def test_two_calls_at_once(W):
    """Every call on a stream of its own, over and over: the bits of one made alone."""
    todo = calls(W, 100)
    want = [c() for c in todo]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in todo]
    got = [[] for _ in todo]
    for _ in range(20):
        for i, (c, s) in enumerate(zip(todo, streams)):
            with torch.cuda.stream(s):
                got[i].append(c())
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        for one in g:
            assert all(torch.equal(x, y) for x, y in zip(one, w))
    W.device_check()


def test_captured_calls(W):
    """Graphs of the same calls replayed in turn and next to eager ones; each has memory of its own."""
    todo = calls(W, 200)
    want = [c() for c in todo]
    graphs, outs = [], []
    for c in todo + todo:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(c())
        graphs.append(g)
    for turn in range(5):
        for o in outs:
            for t in o:
                t.fill_(float("nan"))
        for o in outs:
            o[2].zero_()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            for g in graphs[len(todo):]:
                g.replay()
        for g in graphs[:len(todo)]:
            g.replay()
        eager = [c() for c in todo]
        torch.cuda.synchronize()
        for i, o in enumerate(outs):
            w = want[i % len(todo)]
            assert torch.equal(o[0], w[0]) and torch.equal(o[1], w[1])
            # a graph keeps its zeroed buffer: a replay zeroes it again
            assert torch.equal(o[2], w[2])
        assert all(torch.equal(x, y) for e, w in zip(eager, want) for x, y in zip(e, w))
    W.device_check()


def test_a_captured_decode_loop_grows_with_its_lengths(W):
    """Append, attend and score in one graph; the lengths on the device are all that changes."""
    B, H, share, D, V = 3, 2, 4, 128, 1000
    b = Batch(W, [0] * B, H, D, width=3)
    b.len.zero_()
    rng = np.random.default_rng(5)
    k, v = (torch.empty(B, H, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q = torch.empty(B, H * share, D, dtype=torch.bfloat16, device="cuda")
    logits = torch.randn(B, V, device="cuda")
    mass = torch.zeros(B, H, b.width * 64, device="cuda")

    def step():
        b.len.add_(1)
        W.kv4_append(b.cache, k, v, b.table, b.len)
        out = W.kv4_attend(b.cache, q, b.table, b.len, mass=mass)
        return out, *W.logprobs(logits, top_k=3)[1:]

    step()
    b.len.zero_(), mass.zero_()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out, entropy, top, ids = step()
    ks, vs = [], []
    for n in range(1, 150):
        kn, vn, qn = draw((B, H, D), rng), draw((B, H, D), rng), draw((B, H * share, D), rng)
        k.copy_(dev16(kn)), v.copy_(dev16(vn)), q.copy_(dev16(qn))
        logits.normal_()
        g.replay()
        ks.append(K.held(kn)), vs.append(K.held(vn))
        if n % 16 in (0, 1, 15) or n > 140:
            for i in range(B):
                want, _, _, tol, _, _ = K.attend(f64(qn[i:i + 1]), np.stack([x[i] for x in ks]), np.stack([x[i] for x in vs]),
                                                 D ** -0.5)
                assert (np.abs(f64(bits(out[i:i + 1])) - want) <= tol).all()
        assert torch.equal(ids[:, 0].long(), logits.argmax(1))
    # all the weight of all steps
    assert torch.allclose(mass.sum(2), torch.full((B, H), 149.0 * share, device="cuda"), rtol=1e-5)
    W.device_check()


def test_captured_evictions(W):
    b = Batch(W, [300, 100, 60], 2, 64, width=5, spare=9)
    free = [p for p in range(b.pages) if p not in set(b.table_np.flatten())]
    out = ints(np.array(free[:6]).reshape(3, 2))
    mass = torch.rand(3, 2, 320, device="cuda")
    want = W.kv4_evict(b.cache, b.table, b.len, mass, 90, 7, out)
    starts = starts_of([90, 90, 60])
    want_k = W.kv4_read(b.cache, out, want[0], starts, rows=240)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lengths, m = W.kv4_evict(b.cache, b.table, b.len, mass, 90, 7, out)  # chosen places are the call's own memory
        k, v = W.kv4_read(b.cache, out, lengths, starts, rows=240)
    for _ in range(3):
        for t in (m, k, v):
            t.fill_(3.0)
        lengths.zero_()
        g.replay()
        assert torch.equal(lengths, want[0]) and torch.equal(m, want[1])
        assert torch.equal(k, want_k[0]) and torch.equal(v, want_k[1])
    W.device_check()


def test_pages_past_four_gigabytes(W):
    """Pages at both ends and around 2^32 and 2^33 bytes of a cache of 9.5 GB; tables of a sequence alternate between them."""
    H, D = 8, 128
    page = H * 72 * D
    pages = (19 << 29) // page
    near = [(1 << 32) // page - 1, (1 << 32) // page, (1 << 32) // page + 1, (1 << 33) // page, (1 << 33) // page + 1, pages - 1, 0, 1]
    rng = np.random.default_rng(3)
    lengths = [250, 200]
    b = Batch(W, [0, 0], H, D, width=4)
    b.cache.free()
    b.cache = W.kv4_create(pages, H, D)
    b.table_np = np.array(near, np.int32).reshape(2, 4)
    b.table, b.lengths, b.len = ints(b.table_np), lengths, ints(lengths)
    k, v = draw((450, H, D), rng), draw((450, H, D), rng)
    W.kv4_append(b.cache, dev16(k), dev16(v), b.table, b.len, starts_of(lengths))
    got = W.kv4_read(b.cache, b.table, b.len, starts_of(lengths), rows=450)
    same_values(bits(got[0]), K.held(k))
    same_values(bits(got[1]), K.held(v))
    b.ks, b.vs = [K.held(k[:250]), K.held(k[250:])], [K.held(v[:250]), K.held(v[250:])]
    attend_matches(W, b, draw((2, 2 * H, D), rng), [1, 1])
    mass = torch.rand(2, H, 256, device="cuda")
    out = ints([[pages - 2, pages // 2], [pages // 2 + 1, 5]])
    kept = torch.empty(2, H, 100, dtype=torch.int32, device="cuda")
    n, _ = W.kv4_evict(b.cache, b.table, b.len, mass, 100, 10, out, kept=kept)
    back = f64(bits(W.kv4_read(b.cache, out, n, starts_of([100, 100]), rows=200)[0])).reshape(2, 100, H, D)
    for i in range(2):
        for h in range(H):
            same_values(bits(torch.from_numpy(back[i, :, h]).bfloat16()), b.ks[i][kept[i, h].cpu().numpy(), h])
    W.device_check()
    b.cache.free()


def test_mass_and_rows_past_two_billion_elements(W):
    """Weights of 2^31 places and logits of 2^31 elements: the last rows are right."""
    H, D = 2, 64
    width = 1 << 14
    B = (1 << 31) // (H * width * 64) + 2
    c = W.kv4_create(4, H, D)
    table = torch.zeros(B, width, dtype=torch.int32, device="cuda")
    table[:, 0] = torch.arange(B, device="cuda") % 4
    lengths = torch.zeros(B, dtype=torch.int32, device="cuda")
    lengths[-3:] = 40
    k = dev16(draw((40, H, D), np.random.default_rng(1)))
    for i in range(3):
        W.kv4_append(c, k, k, table[B - 3 + i:B - 2 + i], lengths[-1:], ints([0, 40]))
    mass = torch.zeros(B, H, width * 64, device="cuda")
    q = dev16(draw((B, 4, D), np.random.default_rng(2)))
    W.kv4_attend(c, q, table, lengths, mass=mass)
    assert torch.allclose(mass[-3:, :, :40].sum(2), torch.full((3, H), 2.0, device="cuda"), rtol=1e-5)
    assert not mass[:-3].any() and not mass[-3:, :, 40:].any()
    kept = torch.empty(3, H, 8, dtype=torch.int32, device="cuda")
    out = ints([[0], [1], [2]])
    W.kv4_evict(c, table[-3:].contiguous(), lengths[-3:].contiguous(), mass[-3:], 8, 2, ints([[3], [3], [3]]), kept=kept)
    for i in range(3):
        for h in range(H):
            want = K.evict(mass[B - 3 + i, h, :40].cpu().numpy(), 40, 8, 2)
            assert np.array_equal(kept[i, h].cpu().numpy(), want)
    del mass, out
    V = 20011
    T = (1 << 31) // V + 2
    z = torch.empty(T, V, dtype=torch.bfloat16, device="cuda")
    for i in range(0, T, 8192):
        z[i:i + 8192].normal_(0, 3)
    ids = torch.randint(0, V, (T,), device="cuda")
    lp, _, _, top = W.logprobs(z, ids, 3)
    for i in (0, T // 2, T - 2, T - 1):
        want = torch.log_softmax(z[i].double(), 0)
        assert abs(float(lp[i]) - float(want[ids[i]])) < 1e-5
        assert torch.equal(top[i].long(), torch.sort(z[i].float(), descending=True, stable=True).indices[:3])
    W.device_check()


def test_random_calls_on_three_streams(W):
    """Random shapes, each call on one of three streams at once, every result against the definition."""
    rng = np.random.default_rng(77)
    streams = [torch.cuda.Stream() for _ in range(3)]
    jobs = []
    for n in range(45):
        D, H = int(rng.choice([64, 128, 256])), int(rng.integers(1, 5))
        share = int(rng.choice([1, 2, 3, 4, 6, 8, 11, 17]))
        B = int(rng.integers(1, 7))
        lengths = [int(x) for x in np.exp(rng.uniform(0, 7, B)).astype(int) - 1]
        single = bool(rng.integers(0, 2))
        rows = [1] * B if single else [int(x) for x in rng.integers(0, 6, B)]
        if sum(rows) == 0:
            rows[0] = 1
        window = int(rng.choice([0, 0, 1, 30, 200]))
        with torch.cuda.stream(streams[n % 3]):
            b = Batch(W, lengths, H, D, seed=n)
            q = draw((sum(rows), H * share, D), rng, 1.5)
            lse = torch.empty(sum(rows), H * share, device="cuda")
            mass = torch.zeros(B, H, b.width * 64, device="cuda")
            out = W.kv4_attend(b.cache, dev16(q), b.table, b.len, None if single else starts_of(rows), window=window,
                               lse=lse, mass=mass)
        jobs.append((b, q, rows, window, out, lse, mass))
    torch.cuda.synchronize()
    for b, q, rows, window, out, lse, mass in jobs:
        at = 0
        for i, r in enumerate(rows):
            wo, wl, wm, to, tl, tm = K.attend(f64(q[at:at + r]), b.ks[i], b.vs[i], b.D ** -0.5, window)
            assert (np.abs(f64(bits(out[at:at + r])) - wo) <= to).all()
            seen = ~np.isneginf(wl)
            got = lse[at:at + r].cpu().numpy().astype(np.float64)
            assert np.array_equal(np.isneginf(got), ~seen) and (np.abs(got[seen] - wl[seen]) <= tl[seen]).all()
            n = b.lengths[i]
            assert (np.abs(mass[i, :, :n].cpu().numpy() - wm) <= tm + 1e-7).all()
            at += r
    W.device_check()
