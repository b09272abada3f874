"""4-bit products of every way to spread rows over blocks, on streams next to each other and in graphs.

plan() restates how the library chooses; the shapes below are asserted to take
the path that their test is for.
"""
import pytest

from oracle import q4_moe_oracle as Q

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

WHOLE, CUT, CLUSTERS = "whole", "cut", "clusters"


@pytest.fixture(scope="module")
def W():
    from decode_gemv_sign_gb300 import build, wcomp

    build.build()
    wcomp.lib()
    return wcomp


def plan(N, K, B):
    """Whole units (32 rows) a block, units cut anywhere and joined in memory, or shared by clusters; whether blocks
    prepare x themselves.  In k-steps of 256 columns: a cut costs 40, a cluster 16, a kernel for x 8."""
    ctas = 2 * torch.cuda.get_device_properties(0).multi_processor_count
    units, steps = -(-N // 32), -(-K // 256)

    def at_once(k):
        return -(-k // 8) * 8

    def shared(split, team):
        return B <= 8 and not split and units <= ctas and B * 2 * -(-steps // team) <= 64

    each = -(-units * steps // ctas)
    split = -(-units // ctas) * steps > each + 40
    best = (at_once(each) + 40 if split else at_once(steps) * -(-units // ctas), CUT if split else WHOLE, shared(split, 1))
    best = (best[0] + (0 if best[2] else 8), *best[1:])
    team = 2
    while team <= min(8, steps) and units * team <= ctas:
        x = shared(False, team)
        cost = at_once(-(-steps // team)) + 16 + (0 if x else 8)
        if cost < best[0]:
            best = (cost, CLUSTERS, x)
        team *= 2
    return best[1:]


# N, K, B, how, and whether blocks prepare x themselves
PATHS = [(512, 4096, 2, WHOLE, True), (9728, 2048, 5, WHOLE, False), (9728, 2048, 13, WHOLE, False),
         (512, 8192, 1, CLUSTERS, True), (64, 40000, 8, CLUSTERS, False), (64, 40000, 16, CLUSTERS, False),
         (9744, 14350, 1, CUT, False), (9744, 14350, 8, CUT, False), (9744, 14350, 16, CUT, False)]


class Product:
    """A random weight and x; the reference and its bound in 64 bits on the GPU."""

    def __init__(self, W, N, K, B, group, seed):
        self.N, self.K, self.group = N, K, group
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.codes = torch.randint(0, 256, (N, (K + 1) // 2), dtype=torch.uint8, device="cuda", generator=g)
        self.scales = (torch.rand(N, -(-K // group), device="cuda", generator=g) * 0.02).bfloat16()
        self.x = torch.randn(B, K, device="cuda", generator=g).bfloat16()
        self.c = W.q4_pack(self.codes, self.scales, K, group)

    def check(self, y):
        steps = -(-self.K // self.group) + 64
        for r in range(0, self.N, 1218):
            codes = self.codes[r:r + 1218]
            v = torch.stack([codes & 15, codes >> 4], -1).flatten(1)[:, :self.K].double() - 8
            v *= self.scales[r:r + 1218].double().repeat_interleave(self.group, 1)[:, :self.K]
            want, tol = self.x.double() @ v.T, steps * Q.EPS * (self.x.double().abs() @ v.abs().T)
            assert ((y[:, r:r + 1218].double() - want).abs() <= tol).all()


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("N,K,B,how,x_in_blocks", PATHS)
def test_each_path(W, N, K, B, how, x_in_blocks, group):
    assert plan(N, K, B) == (how, x_in_blocks)
    p = Product(W, N, K, B, group, seed=N + B + group)
    launches = W.launch_count()
    y = W.q4_gemv(p.c, p.x)
    assert W.launch_count() - launches == (1 if x_in_blocks else 2)
    p.check(y)
    assert torch.equal(W.q4_gemv(p.c, p.x), y)
    W.device_check()


def test_paths_on_streams_and_in_graphs(W):
    """Each call has counters, parts and records of its own: two streams and two graphs of all paths at once."""
    products = [Product(W, N, K, B, 64, seed=i) for i, (N, K, B, _, _) in enumerate(PATHS)]
    want = [W.q4_gemv(p.c, p.x) for p in products]
    for p, y in zip(products, want):
        p.check(y)
    graphs = []
    for _ in range(2):
        held, g = [torch.zeros_like(y) for y in want], torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g):
            for p, y in zip(products, held):
                W.q4_gemv(p.c, p.x, y)
        graphs.append((g, held, torch.cuda.Stream()))
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    out = []
    for _ in range(15):
        for g, held, s in graphs:
            with torch.cuda.stream(s):
                for y in held:
                    y.zero_()
                g.replay()
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                order = products if i else products[::-1]
                ys = [W.q4_gemv(p.c, p.x) for p in order]
                out.append(ys if i else ys[::-1])
    torch.cuda.synchronize()
    W.device_check()
    for ys in (*out, *(held for _, held, _ in graphs)):
        assert all(torch.equal(a, b) for a, b in zip(ys, want))
