"""Log probabilities, entropy and top alternatives against their definition in 64 bits.

Indices have to be equal; errors are held to the bound derived in
oracle.kv4_oracle.logprobs and the rounding of the results.
"""
import numpy as np
import pytest

from oracle import kv4_oracle as K
from oracle.q4_moe_oracle import bf16, f64

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def W():
    from decode_gemv_sign_gb300 import build, wcomp

    build.build()
    wcomp.lib()
    return wcomp


def to_device(z, dtype):
    if dtype == "bf16":
        return torch.from_numpy(bf16(z).view(np.int16)).cuda().view(torch.bfloat16), f64(bf16(z))
    z = z.astype(np.float32)
    return torch.from_numpy(z).cuda(), z.astype(np.float64)


def matches(W, logits, z, ids, top_k, scale=1.0):
    T, V = z.shape
    idd = None if ids is None else torch.tensor(ids, dtype=torch.int64, device="cuda")
    lse = torch.empty(T, device="cuda")
    lp, ent, top, top_ids = W.logprobs(logits, idd, top_k, scale=scale, lse=lse)
    wlp, went, wlse, wtop, wids, tol = K.logprobs(z, ids, top_k, scale)
    if top_k == 0:
        assert top is None and top_ids is None
    else:
        assert np.array_equal(top_ids.cpu().numpy(), wids)

    def near(got, want, extra):
        got = got.cpu().numpy().astype(np.float64)
        odd = ~np.isfinite(want)
        assert np.array_equal(got[odd], want[odd], equal_nan=True) and np.isfinite(got[~odd]).all()
        t = np.broadcast_to(tol.reshape(-1, *[1] * (want.ndim - 1)), want.shape) + extra
        assert (np.abs(got - want)[~odd] <= t[~odd]).all(), np.abs(got - want)[~odd].max()

    eps = 2.0 ** -23
    mag = np.where(np.isfinite(z), np.abs(z), 0.0).max(1) * scale  # of the terms that a result is the difference of
    if ids is None:
        assert lp is None
    else:
        near(lp, wlp, 4 * eps * np.abs(np.where(np.isfinite(wlp), wlp, 0)) + 1e-44)
    near(lse, wlse, 4 * eps * mag)
    # a term of the entropy is off by its weight's error times its logarithm
    worst = np.where(np.isfinite(z), z, np.inf)
    spread = np.minimum((np.where(np.isfinite(z), z, -np.inf).max(1) - worst.min(1)) * scale, 100.0)
    with np.errstate(all="ignore"):
        near(ent, went, tol * np.where(np.isfinite(spread), spread, 0) + 8 * eps * np.where(np.isfinite(went), went, 0) + 1e-44)
    if top_k:
        near(top, wtop, (4 * eps * np.abs(np.where(np.isfinite(wtop), wtop, 0))) + 1e-44)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("T,V,k", [(1, 1, 1), (1, 2, 2), (3, 31, 0), (2, 32, 32), (5, 1000, 20), (1, 4097, 64), (7, 8191, 5),
                                   (2, 50001, 8), (1, 151552, 20), (33, 257, 3)])
def test_logprobs_are_the_definition(W, dtype, T, V, k):
    rng = np.random.default_rng(V + T)
    logits, z = to_device(rng.standard_normal((T, V)) * 3, dtype)
    ids = rng.integers(0, V, T)
    ids[0] = V - 1
    matches(W, logits, z, ids.tolist(), k)
    matches(W, logits, z, None, k, scale=0.3)
    matches(W, logits, z, ids.tolist(), 0, scale=4.0)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_strided_and_unaligned_rows(W, dtype):
    rng = np.random.default_rng(4)
    whole, z = to_device(rng.standard_normal((6, 2007)) * 2, dtype)
    for lo, hi in ((0, 2007), (1, 2007), (3, 1500), (8, 2000), (5, 6), (2, 5)):
        part, zp = whole[:, lo:hi], z[:, lo:hi]
        matches(W, part, zp, [0] * 6, min(4, hi - lo))
        matches(W, part[1:2], zp[1:2], [hi - lo - 1], 1)
        matches(W, part[::2], zp[::2], [0] * 3, 1)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("V", [100, 9000])
def test_masked_vocabularies(W, dtype, V):
    """Rows with few tokens left, one, none; masks of -inf and of the type's lowest value; ties everywhere."""
    rng = np.random.default_rng(V)
    lowest = -3.3895313892515355e38 if dtype == "bf16" else -3.4028234663852886e38
    z = rng.standard_normal((9, V))
    z[0, 5:] = -np.inf
    z[1, :] = -np.inf
    z[2, :-1] = -np.inf
    z[3, 3:] = lowest
    z[4, :] = lowest
    z[5, :] = 1.0
    z[6, ::2] = 0.0
    z[6, 1::2] = -0.0
    z[7, 7] = 60.0
    z[8, V // 2] = -1e30
    logits, zv = to_device(z, dtype)
    matches(W, logits, zv, [0, 0, V - 1, 1, V - 1, 50, 3, 7, V // 2], 20)
    matches(W, logits[:3], zv[:3], [7, V - 1, 0], 64)


def test_values_that_are_not_numbers(W):
    rng = np.random.default_rng(1)
    z = rng.standard_normal((6, 3000))
    z[0, 2999] = np.nan
    z[1, :] = np.nan
    z[2, 5] = np.inf
    z[3, [7, 8]] = np.inf
    z[4, 0], z[4, 1] = np.nan, np.inf
    logits, zv = to_device(z, "fp32")
    matches(W, logits, zv, [0, 1, 5, 6, 7, 8], 5)


def test_small_entropies_keep_their_bits(W):
    """One token far above the others: entropy and its distance from probability 1 to relative precision."""
    z = np.zeros((5, 70000))
    z[:, 123] = [15.0, 25.0, 40.0, 60.0, 80.0]
    logits, zv = to_device(z, "fp32")
    lp, ent, top, _ = W.logprobs(logits, torch.full((5,), 123, device="cuda"), 1)
    s = 69999 * np.exp(-z[:, 123])
    want, went = -np.log1p(s), np.log1p(s) + s * z[:, 123] / (1 + s)
    for got, w in ((lp, want), (top[:, 0], want), (ent, went)):
        assert (np.abs(got.cpu().numpy() / w - 1) < 70000 / 128 * K.EPS + 1e-6).all()


def test_given_tokens_outside_the_vocabulary(W):
    logits, z = to_device(np.random.default_rng(2).standard_normal((6, 50)), "fp32")
    matches(W, logits, z, [-1, -100, 50, 2 ** 31, -2 ** 63, 2 ** 62], 0)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_ties_go_to_the_lowest_index(W, dtype):
    rng = np.random.default_rng(3)
    logits, z = to_device(rng.integers(-3, 4, (8, 20000)).astype(float), dtype)
    matches(W, logits, z, [0] * 8, 64)
    z2 = np.full((2, 5000), -1.0)
    z2[0, 4900:] = 2.0
    z2[1, ::50] = 2.0
    logits, z2 = to_device(z2, dtype)
    matches(W, logits, z2, [0] * 2, 64)


def test_many_rows_repeat_bit_for_bit(W):
    g = torch.Generator(device="cuda").manual_seed(5)
    logits = torch.randn(3000, 777, device="cuda", generator=g)
    ids = torch.randint(0, 777, (3000,), device="cuda", generator=g)
    a, b = W.logprobs(logits, ids, 7), W.logprobs(logits, ids, 7)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    want = torch.log_softmax(logits.double(), 1)
    assert (a[0].double() - want.gather(1, ids[:, None])[:, 0]).abs().max() < 1e-5
    assert torch.equal(a[3].long(), torch.sort(logits, dim=1, descending=True, stable=True).indices[:, :7])
    alone = W.logprobs(logits[17:18], ids[17:18], 7)
    assert torch.equal(alone[3][0], a[3][17]) and abs(float(alone[0][0] - a[0][17])) < 1e-5


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_long_rows_by_one_block(W, dtype):
    """Rows too many to be shared, and longer than one batch for each of a block's buckets."""
    T, V = 310, 300007
    g = torch.Generator(device="cuda").manual_seed(6)
    logits = (torch.randn(T, V, device="cuda", generator=g) * 3).to(torch.float32 if dtype == "fp32" else torch.bfloat16)
    logits[3] = 1.0
    logits[4, :V - 70] = float("-inf")
    ids = torch.randint(V - 70, V, (T,), device="cuda", generator=g)
    lp, _, top, top_ids = W.logprobs(logits, ids, 64)
    pick = [0, 1, 2, 3, 4, 151, 152, 303, 304, 309]
    some = logits[pick].double()
    order = torch.sort(logits[pick].float(), dim=1, descending=True, stable=True).indices[:, :64]
    assert torch.equal(top_ids[pick].long(), order)
    want = torch.log_softmax(some, 1)
    assert (lp[pick].double() - want.gather(1, ids[pick, None])[:, 0]).abs().max() < 1e-5
    assert (top[pick].double() - want.gather(1, order)).abs().max() < 1e-5


def test_no_rows(W):
    lp, ent, top, ids = W.logprobs(torch.empty(0, 10, device="cuda"), torch.empty(0, dtype=torch.int64, device="cuda"), 3)
    assert lp.shape == ent.shape == (0,) and top.shape == ids.shape == (0, 3)


def test_python_refusals(W):
    z = torch.zeros(2, 10, device="cuda")
    for call, err in ((lambda: W.logprobs(z.double()), TypeError), (lambda: W.logprobs(z[0]), ValueError),
                      (lambda: W.logprobs(z[:, ::2]), ValueError), (lambda: W.logprobs(z, top_k=11), ValueError),
                      (lambda: W.logprobs(z, top_k=-1), ValueError),
                      (lambda: W.logprobs(z, torch.zeros(2, device="cuda")), ValueError),
                      (lambda: W.logprobs(z, torch.zeros(3, dtype=torch.int64, device="cuda")), ValueError),
                      (lambda: W.logprobs(z, torch.zeros(2, dtype=torch.int64)), ValueError),
                      (lambda: W.logprobs(z, scale=0.0), W.WcompError),
                      (lambda: W.logprobs(z[:1].expand(2, 10)), W.WcompError),
                      (lambda: W.logprobs(torch.zeros(1, 100, device="cuda"), top_k=65), W.WcompError)):
        with pytest.raises(err):
            call()
