"""4-bit weights with group scales against their definition in 64 bits.

Codes, scales and read-back values have to be equal bit for bit; the GEMV is
held to the error that its fp32 sums can make (derived in oracle.q4_moe_oracle.gemv).
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
    return torch.from_numpy(np.ascontiguousarray(a).view(np.int16)).cuda()


def bits(t):
    return t.view(torch.int16).cpu().numpy().view(np.uint16)


def draw(N, K, seed, M=None):
    spec = synth.WeightSpec("q4", N * (M or 1), K, "t4", 0.02, 0.001, "normal", 0.1, seed=seed)
    w = synth.gen_weights_np(spec)
    return w if M is None else w.reshape(M, N, K)


def same_held(W, c, w, group):
    """The held codes and scales, and the values read back, are the definition's."""
    codes, scales = Q.q4_encode(w, group)
    got_codes, got_scales = W.q4_unpack(c)
    assert np.array_equal(got_codes.cpu().numpy(), Q.pack_codes(codes))
    assert np.array_equal(bits(got_scales), scales)
    out = bits(W.q4_decode(c))
    want = Q.bf16(Q.q4_values(codes, scales, group))
    zero = (want & 0x7FFF) == 0  # the sign of a zero is not specified
    nan = (want & 0x7FFF) > 0x7F80
    assert np.array_equal(out[~zero & ~nan], want[~zero & ~nan])
    assert ((out[zero] & 0x7FFF) == 0).all() and ((out[nan] & 0x7FFF) > 0x7F80).all()


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("shape", [(1, 1), (1, 31), (16, 128), (17, 129), (33, 257), (5, 1000), (48, 2048), (100, 77)])
def test_encode_is_the_definition(W, shape, group):
    w = draw(*shape, seed=sum(shape) + group)
    c = W.q4_encode(dev(w), group)
    assert c.info()["N"] == shape[0] and c.info()["K"] == shape[1] and c.info()["group"] == group
    same_held(W, c, w, group)


@pytest.mark.parametrize("group", [32, 64, 128])
def test_every_bf16_value_against_many_scales(W, group):
    """Every positive finite BF16 value as a group's largest, next to values around each rounding edge."""
    tops = np.arange(1, 0x7F80, dtype=np.uint16)
    rows = np.zeros((len(tops), group), np.uint16)
    rng = np.random.default_rng(1)
    scale = Q.f64(Q.bf16(Q.f64(tops) / 7.0))
    for i in range(1, group):
        # halves of the scale and their neighbours, both signs
        v = Q.bf16(scale * (rng.integers(-13, 14, len(tops)) / 2.0)).astype(np.int64)
        v = v + rng.integers(-1, 2, len(tops))
        v = np.clip(v & 0x7FFF, 0, tops) | (v & 0x8000)
        rows[:, i] = v.astype(np.uint16)
    rows[:, 0] = tops
    c = W.q4_encode(dev(rows), group)
    same_held(W, c, rows, group)


def test_non_finite_and_zero_groups(W):
    w = draw(20, 300, 9)
    w[3, 5] = 0x7F80    # inf
    w[4, 200] = 0xFF80  # -inf
    w[5, 299] = 0x7FC1  # NaN
    w[6, 128:256] = 0   # a group of zeros
    w[7, :] = 0x8000    # a row of -0
    w[8, 0:128] = 1     # the smallest subnormal: the scale underflows to zero
    for group in (32, 64, 128):
        c = W.q4_encode(dev(w), group)
        same_held(W, c, w, group)
        x = synth.gen_x_np(3, 300, 4)
        y = W.q4_gemv(c, dev(x)).cpu().numpy()
        bad = np.zeros(20, bool)
        bad[3:6] = True
        assert np.isnan(y[:, bad]).all() and np.isfinite(y[:, ~bad]).all()
        assert (y[:, 7] == 0).all()


@pytest.mark.parametrize("offset", [1, 3, 8])
def test_encode_and_decode_of_unaligned_tensors(W, offset):
    w = draw(9, 256, 21)
    buf = torch.zeros(9 * 256 + offset, dtype=torch.int16, device="cuda")
    view = buf[offset:].view(9, 256)
    view.copy_(dev(w))
    c = W.q4_encode(view, 64)
    same_held(W, c, w, 64)
    out = torch.zeros(9 * 256 + offset + 8, dtype=torch.int16, device="cuda")
    W.q4_decode(c, out[offset:offset + 9 * 256].view(9, 256))
    codes, scales = Q.q4_encode(w, 64)
    got = out.cpu().numpy().view(np.uint16)
    assert np.array_equal(Q.f64(got[offset:offset + 9 * 256]), Q.f64(Q.bf16(Q.q4_values(codes, scales, 64))).reshape(-1))
    assert not got[:offset].any() and not got[offset + 9 * 256:].any()


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("shape", [(7, 64), (16, 4096), (40, 333)])
def test_pack_round_trips_every_code(W, shape, group):
    """Codes quantised elsewhere (0 included) and any scale come back as they went in."""
    N, K = shape
    rng = np.random.default_rng(N)
    codes = rng.integers(0, 16, (2, N, K)).astype(np.uint8)
    scales = rng.integers(0, 1 << 16, (2, N, -(-K // group))).astype(np.uint16)
    c = W.q4_pack(torch.from_numpy(Q.pack_codes(codes)).cuda(), dev(scales).view(torch.bfloat16), K, group)
    assert c.shape == (2, N, K)
    got_codes, got_scales = W.q4_unpack(c)
    assert np.array_equal(got_codes.cpu().numpy(), Q.pack_codes(codes))
    assert np.array_equal(bits(got_scales), scales)


@pytest.mark.parametrize("B", [1, 2, 7, 8, 9, 16])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("shape", [(1, 1), (1, 5000), (15, 130), (16, 128), (300, 2048), (37, 1001), (2050, 272),
                                   (130, 8192)])
def test_gemv(W, shape, group, B):
    N, K = shape
    rng = np.random.default_rng(N + K + B)
    codes = rng.integers(0, 16, (N, K)).astype(np.uint8)
    scales = Q.bf16(rng.uniform(0.001, 0.02, (N, -(-K // group))))
    c = W.q4_pack(torch.from_numpy(Q.pack_codes(codes)).cuda(), dev(scales).view(torch.bfloat16), K, group)
    x = synth.gen_x_np(B, K, N + B)
    want, tol = Q.gemv(Q.q4_values(codes, scales, group), x, group)
    y = torch.full((B, N), float("nan"), device="cuda")
    W.q4_gemv(c, dev(x), y)
    assert (np.abs(y.cpu().numpy() - want) <= tol).all()
    assert torch.equal(W.q4_gemv(c, dev(x)), y)  # the same bits again
    W.device_check()


@pytest.mark.parametrize("B", [1, 16])
def test_gemv_one_hot_reads_every_column(W, B):
    """x = one column of ones: y is that column, exactly."""
    N, K, group = 50, 400, 32
    w = draw(N, K, 3)
    c = W.q4_encode(dev(w), group)
    v = Q.q4_values(*Q.q4_encode(w, group), group)
    for k0 in range(0, K, B):
        x = np.zeros((B, K), np.uint16)
        x[np.arange(B), k0 + np.arange(B)] = 0x3F80
        assert np.array_equal(W.q4_gemv(c, dev(x)).cpu().numpy().astype(np.float64), v[:, k0:k0 + B].T)


def test_gemv_of_unaligned_x_and_row_slices(W):
    N, K = 64, 512
    w = draw(N, K, 5)
    c = W.q4_encode(dev(w), 64)
    x = synth.gen_x_np(3, K, 8)
    want = W.q4_gemv(c, dev(x))
    for off in (1, 8, 16):
        buf = torch.zeros(3 * K + off, dtype=torch.int16, device="cuda")
        buf[off:].copy_(dev(x).view(-1))
        assert torch.equal(W.q4_gemv(c, buf[off:].view(3, K)), want)
    # one row of a larger batch, 1-D
    assert torch.equal(W.q4_gemv(c, dev(x)[1]), want[1:2])


def test_gemv_infinite_and_nan_x_stay_in_their_row(W):
    N, K = 40, 700
    w = draw(N, K, 6)
    c = W.q4_encode(dev(w), 32)
    x = synth.gen_x_np(12, K, 9)
    clean = W.q4_gemv(c, dev(x))
    x[4, 13] = 0x7FC0
    y = W.q4_gemv(c, dev(x))
    assert torch.isnan(y[4]).all()
    keep = [b for b in range(12) if b != 4]
    assert torch.equal(y[keep], clean[keep])


def test_gemv_infinite_x_has_the_weights_signs(W):
    N, K, group = 40, 700, 64
    codes = np.random.default_rng(3).integers(0, 16, (N, K)).astype(np.uint8)
    scales = Q.bf16(np.full((N, -(-K // group)), 0.01))
    c = W.q4_pack(torch.from_numpy(Q.pack_codes(codes)).cuda(), dev(scales).view(torch.bfloat16), K, group)
    x = synth.gen_x_np(10, K, 9)
    x[0, 130], x[9, 699] = 0x7F80, 0xFF80
    y = W.q4_gemv(c, dev(x)).cpu().numpy()
    for b, col, sign in ((0, 130, 1), (9, 699, -1)):
        v = codes[:, col].astype(int) - 8
        want = np.where(v == 0, np.nan, np.inf * sign * np.sign(v + (v == 0)))
        assert np.array_equal(y[b], want.astype(np.float32), equal_nan=True)
    assert np.isfinite(y[1:9]).all()


@pytest.mark.parametrize("off", [0, 1, 2, 4])
@pytest.mark.parametrize("B,K", [(1, 8192), (1, 8193), (1, 8190), (8, 1024), (8, 1025), (3, 2559), (5, 1), (2, 258)])
def test_gemv_around_the_most_x_that_blocks_prepare_themselves(W, B, K, off):
    """Up to 64 blocks of 128 columns of x, from any alignment, with an infinity in its row and nowhere else."""
    N, group = 100, 128
    w = draw(N, K, seed=K)
    c = W.q4_encode(dev(w), group)
    x = synth.gen_x_np(B, K, B + off)
    want, tol = Q.gemv(Q.q4_values(*Q.q4_encode(w, group), group), x, group)
    buf = torch.full((B * K + off + 8,), 0x7F80, dtype=torch.int16, device="cuda")
    view = buf[off:off + B * K].view(B, K)
    view.copy_(dev(x))
    assert (np.abs(W.q4_gemv(c, view).cpu().numpy() - want) <= tol).all()
    view[B - 1, K - 1] = 0x7FC0
    y = W.q4_gemv(c, view).cpu().numpy()
    assert np.isnan(y[B - 1]).all() and (np.abs(y[:B - 1] - want[:B - 1]) <= tol[:B - 1]).all()


@pytest.mark.parametrize("B", [1, 7, 13])
@pytest.mark.parametrize("shape", [(32, 40576), (257, 20000), (1000, 9001), (2000, 16300), (4800, 8200)])
def test_gemv_of_few_long_rows(W, shape, B):
    """Fewer tiles than thread blocks: clusters share them, or their sums are cut along the rows and joined."""
    N, K = shape
    w = draw(N, K, seed=N)
    for group in (32, 128):
        c = W.q4_encode(dev(w), group)
        x = synth.gen_x_np(B, K, B)
        want, tol = Q.gemv(Q.q4_values(*Q.q4_encode(w, group), group), x, group)
        y = W.q4_gemv(c, dev(x))
        assert (np.abs(y.cpu().numpy() - want) <= tol).all()
        assert torch.equal(W.q4_gemv(c, dev(x)), y)
    W.device_check()


@pytest.mark.parametrize("B", [1, 8, 11])
def test_gemv_with_rows_cut_over_blocks(W, B):
    """A few more tiles than blocks and long rows: every block takes the same number of columns, rows are joined in
    memory.  The definition in 64 bits on the GPU, by elementary operations."""
    N, K, group = 9744, 14350, 64
    g = torch.Generator(device="cuda")
    g.manual_seed(B)
    codes = torch.randint(0, 256, (N, K // 2), dtype=torch.uint8, device="cuda", generator=g)
    scales = (torch.rand(N, -(-K // group), device="cuda", generator=g) * 0.02).bfloat16()
    x = torch.randn(B, K, device="cuda", generator=g).bfloat16()
    c = W.q4_pack(codes, scales, K, group)
    y = W.q4_gemv(c, x)
    assert torch.equal(W.q4_gemv(c, x), y)
    W.device_check()
    steps = -(-K // group) + 64
    for r in range(0, N, 1218):
        v = torch.stack([codes[r:r + 1218] & 15, codes[r:r + 1218] >> 4], -1).flatten(1).double() - 8
        v *= scales[r:r + 1218].double().repeat_interleave(group, 1)[:, :K]
        want, tol = x.double() @ v.T, steps * Q.EPS * (x.double().abs() @ v.abs().T)
        assert ((y[:, r:r + 1218].double() - want).abs() <= tol).all()


@pytest.mark.parametrize("B", [1, 10])
def test_gemv_of_x_over_a_wide_range(W, B):
    """Magnitudes from 2^-100 to 2^100 in one row: a value keeps its 8 bits down to 2^-31 of the largest of its 128
    columns, and errs by at most 2^-39 of that below."""
    N, K, group = 70, 1100, 32
    rng = np.random.default_rng(B)
    w = draw(N, K, seed=77)
    c = W.q4_encode(dev(w), group)
    x = Q.bf16(rng.standard_normal((B, K)) * 2.0 ** rng.integers(-100, 101, (B, K)))
    x[0, :128] = 0
    v = Q.q4_values(*Q.q4_encode(w, group), group)
    want, tol = Q.gemv(v, x, group)
    xv = np.abs(Q.f64(x))
    for k in range(0, K, 128):
        tol = tol + 2.0 ** -39 * xv[:, k:k + 128].max(1, keepdims=True) * np.abs(v[:, k:k + 128]).sum(1)
    assert (np.abs(W.q4_gemv(c, dev(x)).cpu().numpy() - want) <= tol).all()


def test_calls_on_two_streams_do_not_disturb_each_other(W):
    """Split sums take their own counters and workspace per call."""
    N, K, B = 4096, 4096, 16
    c = W.q4_encode(dev(draw(N, K, 11)), 128)
    xs = [dev(synth.gen_x_np(B, K, 30 + i)) for i in range(2)]
    want = [W.q4_gemv(c, x) for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(W.q4_gemv(c, xs[i]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(y, want[i]) for y in got[i])


def test_gemv_in_a_graph(W):
    N, K, B = 1024, 2048, 12
    c = W.q4_encode(dev(draw(N, K, 12)), 64)
    x = dev(synth.gen_x_np(B, K, 1))
    y = torch.zeros(B, N, device="cuda")
    W.q4_gemv(c, x, y)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        W.q4_gemv(c, x, y)
    x.copy_(dev(synth.gen_x_np(B, K, 2)))
    for _ in range(3):
        y.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, W.q4_gemv(c, x))


def test_refusals(W):
    w = dev(draw(4, 64, 1))
    for group in (0, 16, 96, 256):
        with pytest.raises(W.WcompError):
            W.q4_encode(w, group)
    with pytest.raises(TypeError):
        W.q4_encode(torch.zeros(4, 64, device="cuda"))
    with pytest.raises(ValueError):
        W.q4_encode(w.view(-1))
    with pytest.raises(ValueError):
        W.q4_encode(w.t())
    with pytest.raises(W.WcompError):
        W.q4_encode(torch.zeros(0, 64, dtype=torch.int16, device="cuda"))
    codes = torch.zeros(4, 32, dtype=torch.uint8, device="cuda")
    scales = torch.zeros(4, 2, dtype=torch.bfloat16, device="cuda")
    for bad in ((codes, scales, 66, 32), (codes, scales, 64, 64), (codes, scales, 64, 48)):
        with pytest.raises(ValueError):
            W.q4_pack(*bad)
    with pytest.raises(TypeError):
        W.q4_pack(codes.cpu(), scales, 64, 32)
    with pytest.raises(TypeError):
        W.q4_pack(codes, scales.float(), 64, 32)
    c = W.q4_encode(w, 32)
    x = torch.zeros(17, 64, dtype=torch.int16, device="cuda")
    with pytest.raises(W.WcompError):
        W.q4_gemv(c, x)
    with pytest.raises(ValueError):
        W.q4_gemv(c, x[:2, :32].contiguous())
    with pytest.raises(ValueError):
        W.q4_gemv(c, x[:1], torch.zeros(1, 4, dtype=torch.float64, device="cuda"))
    with pytest.raises(ValueError):
        W.q4_gemv(W.q4_encode(w.view(2, 2, 64), 32), x[:1])
    with pytest.raises(ValueError):
        W.q4_decode(c, torch.zeros(4, 63, dtype=torch.int16, device="cuda"))
    c.free()
    c.free()
    with pytest.raises(ValueError):
        W.q4_gemv(c, x[:1])
