"""Every output of the 4-bit and expert calls between guard words, at sizes that end inside tiles and blocks."""
import numpy as np
import pytest

from decode_gemv_sign_gb300 import synth
from oracle import q4_moe_oracle as Q
from test_gpu_q4 import dev, draw

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

GUARD = 4096  # bytes before and after an output
PATTERN = 0xA5


@pytest.fixture(scope="module")
def W():
    from decode_gemv_sign_gb300 import build, wcomp

    build.build()
    wcomp.lib()
    return wcomp


class Guarded:
    """A contiguous tensor inside a buffer of pattern bytes, `off` elements past the guard."""

    def __init__(self, shape, dtype, off=0):
        size = torch.empty(0, dtype=dtype).element_size()
        self.n, self.at = int(np.prod(shape)) * size, GUARD + off * size
        self.buf = torch.full((self.at + self.n + GUARD,), PATTERN, dtype=torch.uint8, device="cuda")
        self.t = self.buf[self.at:self.at + self.n].view(dtype).view(shape)

    def check(self):
        assert (self.buf[:self.at] == PATTERN).all() and (self.buf[self.at + self.n:] == PATTERN).all()
        return self.t


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("shape", [(1, 1), (31, 255), (33, 257), (17, 1001), (2, 45, 130), (1, 40000)])
def test_unpack_and_decode(W, shape, group):
    w = draw(*shape[-2:], seed=sum(shape), M=shape[0] if len(shape) == 3 else None)
    c = W.q4_encode(dev(w), group)
    codes, scales = Q.q4_encode(w, group)
    K = shape[-1]
    for off in (0, 1):
        a = Guarded((*shape[:-1], (K + 1) // 2), torch.uint8, off)
        b = Guarded((*shape[:-1], -(-K // group)), torch.int16, off)
        assert W.lib().wcomp_q4_unpack(c.handle, a.t.data_ptr(), b.t.data_ptr(), W._stream()) == W.OK
        assert np.array_equal(a.check().cpu().numpy(), Q.pack_codes(codes))
        assert np.array_equal(b.check().cpu().numpy().view(np.uint16), scales)
        out = Guarded(shape, torch.int16, off)
        W.q4_decode(c, out.t)
        want = Q.bf16(Q.q4_values(codes, scales, group))
        assert np.array_equal(Q.f64(out.check().cpu().numpy().view(np.uint16)), Q.f64(want))


@pytest.mark.parametrize("B", [1, 5, 8, 9, 16])
@pytest.mark.parametrize("shape", [(1, 1), (31, 255), (33, 257), (65, 9001), (257, 20000), (5001, 700)])
def test_gemv(W, shape, B):
    N, K = shape
    w = draw(N, K, seed=N + B)
    for group in (32, 128):
        c = W.q4_encode(dev(w), group)
        x = synth.gen_x_np(B, K, N + B)
        want, tol = Q.gemv(Q.q4_values(*Q.q4_encode(w, group), group), x, group)
        for off in (0, 1):
            y = Guarded((B, N), torch.float32, off)
            W.q4_gemv(c, dev(x), y.t)
            assert (np.abs(y.check().cpu().numpy() - want) <= tol).all()
    W.device_check()


@pytest.mark.parametrize("form", ["bf16", 32, 128])
@pytest.mark.parametrize("T,E,k,H,F", [(1, 1, 1, 1, 1), (3, 5, 2, 33, 31), (16, 7, 3, 257, 65), (9, 4, 4, 264, 520), (5, 40, 16, 1001, 333),
                                       (1, 2, 1, 8192, 40), (16, 300, 8, 72, 8)])
def test_moe(W, T, E, k, H, F, form):
    g = torch.Generator(device="cuda")
    g.manual_seed(H + T)

    def bf(*shape):
        return (torch.randn(*shape, device="cuda", generator=g) * 0.1).bfloat16()

    experts = [bf(E, F, H), bf(E, F, H), bf(E, H, F)]
    if form != "bf16":
        experts = [W.q4_encode(w, form) for w in experts]
    x, router = bf(T, H) * 10, bf(E, H)
    ids, weights = torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda")
    want = W.moe(x, router, *experts, k, ids=ids, weights=weights)
    for off in (0, 1):
        y, i, v = Guarded((T, H), torch.bfloat16, off), Guarded((T, k), torch.int32, off), Guarded((T, k), torch.float32, off)
        W.moe(x, router, *experts, k, y=y.t, ids=i.t, weights=v.t)
        assert torch.equal(y.check(), want) and torch.equal(i.check(), ids) and torch.equal(v.check(), weights)
    W.device_check()
