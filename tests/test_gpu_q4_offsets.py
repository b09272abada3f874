"""4-bit weights of more than 2^32 values: quantised, read back, multiplied with, and as experts."""
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


def values(codes, scales, K, group):
    v = torch.stack([codes & 15, codes >> 4], -1).flatten(-2)[..., :K].double() - 8
    return v * scales.double().repeat_interleave(group, -1)[..., :K]


@pytest.mark.parametrize("K", [8192, 8197])
def test_one_matrix(W, K):
    """540000 rows: the last ones against the definition, from the plain layout and from BF16."""
    N, group, last = 540_000, 128, 1000
    assert (N - last) * K > 2 ** 32
    g = torch.Generator(device="cuda")
    g.manual_seed(K)
    codes = torch.randint(0, 256, (N, (K + 1) // 2), dtype=torch.uint8, device="cuda", generator=g)
    if K % 2:
        codes[:, -1] = (codes[:, -1] & 15) | 0x80
    scales = (torch.rand(N, -(-K // group), device="cuda", generator=g) * 0.02).bfloat16()
    c = W.q4_pack(codes, scales, K, group)
    got = W.q4_unpack(c)
    assert torch.equal(got[0], codes) and torch.equal(got[1].view(torch.int16), scales.view(torch.int16))
    del got
    v = values(codes[-last:], scales[-last:], K, group)
    steps = -(-K // group) + 64
    for B in (1, 16):
        x = torch.randn(B, K, device="cuda", generator=g).bfloat16()
        y = W.q4_gemv(c, x)[:, -last:].double()
        assert ((y - x.double() @ v.T).abs() <= steps * Q.EPS * (x.double().abs() @ v.abs().T)).all()
    w = W.q4_decode(c).view(torch.bfloat16)
    # a value of 4 + 8 significant bits, rounded once
    assert ((w[-last:].double() - v).abs() <= 2.0 ** -8 * v.abs()).all()
    c.free()
    again = W.q4_encode(w, group)
    codes2, scales2 = W.q4_unpack(again)
    few = W.q4_encode(w[-last:].contiguous(), group)
    want = W.q4_unpack(few)
    assert torch.equal(codes2[-last:], want[0]) and torch.equal(scales2[-last:].view(torch.int16), want[1].view(torch.int16))
    W.device_check()


def test_experts(W):
    """The last of 70 experts of 8192 x 8192 lies past 2^32 values in each of the three weights."""
    E, H, F, group = 70, 8192, 8192, 64
    assert (E - 1) * H * F > 2 ** 32
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    codes = torch.full((E, F, H // 2), 0x88, dtype=torch.uint8, device="cuda")
    codes[E - 1] = torch.randint(0, 256, (F, H // 2), dtype=torch.uint8, device="cuda", generator=g)
    scales = torch.full((E, F, H // group), 0.002, dtype=torch.bfloat16, device="cuda")
    held = W.q4_pack(codes, scales, H, group)
    x = torch.randn(1, H, device="cuda", generator=g).bfloat16()
    router = torch.zeros(E, H, dtype=torch.bfloat16, device="cuda")
    bias = torch.zeros(E, device="cuda")
    bias[E - 1] = 1.0
    y = W.moe(x, router, held, held, held, 1, bias=bias)
    v = values(codes[E - 1], scales[E - 1], H, group)
    a = v @ x[0].double()
    h = a / (1 + torch.exp(-a)) * a
    want = v @ h
    # one BF16 rounding, and 11 bits of every hidden value
    assert ((y[0].double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -11 * (v.abs() @ h.abs())).all()
    W.device_check()
