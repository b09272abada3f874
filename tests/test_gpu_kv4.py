"""The 4-bit key/value cache, attention over it and eviction from it against their definitions in 64 bits.

What is held has to be equal bit for bit; attention is held to the error bounds
derived in oracle.kv4_oracle.attend; an eviction's choice and copies are exact.
"""
import ctypes

import numpy as np
import pytest

from oracle import kv4_oracle as K
from oracle.q4_moe_oracle import bf16, f64

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

GUARD = 4096


@pytest.fixture(scope="module")
def W():
    from decode_gemv_sign_gb300 import build, wcomp

    build.build()
    wcomp.lib()
    return wcomp


def dev16(a):
    return torch.from_numpy(np.ascontiguousarray(a).view(np.int16)).cuda().view(torch.bfloat16)


def bits(t):
    return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def starts_of(rows):
    return ints(np.concatenate([[0], np.cumsum(rows)]))


def draw(shape, rng, sigma=1.0):
    return bf16(rng.standard_normal(shape) * sigma)


def same_values(got, want):
    """BF16 bits of read-back values are those of the 64-bit values, zeros of either sign alike."""
    want = bf16(want)
    zero = (want & 0x7FFF) == 0
    nan = (want & 0x7FFF) > 0x7F80
    assert np.array_equal(got[~zero & ~nan], want[~zero & ~nan])
    assert ((got[zero] & 0x7FFF) == 0).all() and ((got[nan] & 0x7FFF) > 0x7F80).all()


class Batch:
    """Sequences of the given lengths in a cache, their pages in random order among spare ones."""

    def __init__(self, W, lengths, H, D, seed=0, spare=3, width=None, k=None, v=None):
        self.W, self.lengths, self.H, self.D = W, list(lengths), H, D
        rng = np.random.default_rng(seed)
        need = max(1, max(-(-n // 64) for n in lengths))
        self.width = need + 1 if width is None else width
        B = len(self.lengths)
        self.pages = B * self.width + spare
        self.table_np = rng.permutation(self.pages)[:B * self.width].reshape(B, self.width).astype(np.int32)
        self.table, self.len = ints(self.table_np), ints(self.lengths)
        total = sum(self.lengths)
        self.k = draw((total, H, D), rng) if k is None else k
        self.v = draw((total, H, D), rng) if v is None else v
        self.cache = W.kv4_create(self.pages, H, D)
        if total:
            W.kv4_append(self.cache, dev16(self.k), dev16(self.v), self.table, self.len, starts_of(self.lengths))
        at = np.concatenate([[0], np.cumsum(self.lengths)])
        self.ks = [K.held(self.k[a:b]) for a, b in zip(at, at[1:])]
        self.vs = [K.held(self.v[a:b]) for a, b in zip(at, at[1:])]

    def everything(self):
        return self.W.kv4_read(self.cache, self.table, self.len, starts_of(self.lengths), rows=sum(self.lengths))


# ---------------------------------------------------------------------------
# Writing and reading.
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("lengths", [[1], [64], [65, 0, 1, 63, 64, 130], [0, 200, 7]])
def test_append_and_read_are_the_definition(W, D, lengths):
    b = Batch(W, lengths, 3, D, seed=D + len(lengths))
    k, v = b.everything()
    same_values(bits(k), K.held(b.k))
    same_values(bits(v), K.held(b.v))
    W.device_check()


@pytest.mark.parametrize("D", [64, 128, 256])
def test_tokens_one_by_one_are_the_tokens_at_once(W, D):
    """Decode steps over three sequences give the same cache as one call, bit for bit."""
    lengths = [70, 1, 129]
    whole = Batch(W, lengths, 2, D, seed=5)
    other = W.kv4_create(whole.pages, 2, D)
    at = np.concatenate([[0], np.cumsum(lengths)])
    for step in range(max(lengths)):
        rows = [at[i] + step if step < n else at[i] for i, n in enumerate(lengths)]
        now = [step + 1 if step < n else 0 for n in lengths]  # a finished sequence's row has no place
        W.kv4_append(other, dev16(whole.k[rows]), dev16(whole.v[rows]), whole.table, ints(now))
    a = whole.everything()
    b = W.kv4_read(other, whole.table, whole.len, starts_of(lengths), rows=sum(lengths))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    W.device_check()


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("chunk", [1, 7, 16, 33, 100, 400])
def test_prompts_in_parts_are_the_prompts_at_once(W, D, chunk):
    """Every chunk of up to `chunk` rows a sequence, few or many, from and to any place of a page; rows of nobody behind."""
    lengths = [300, 1, 64, 129, 15]
    whole = Batch(W, lengths, 3, D, seed=6)
    other = W.kv4_create(whole.pages, 3, D)
    at = np.concatenate([[0], np.cumsum(lengths)])
    for step in range(0, max(lengths), chunk):
        now = [min(n, step + chunk) for n in lengths]
        rows = [max(0, n - step) for n in now]
        pick = np.concatenate([np.arange(at[i] + step, at[i] + step + r) for i, r in enumerate(rows)] + [np.zeros(3, int)])
        W.kv4_append(other, dev16(whole.k[pick]), dev16(whole.v[pick]), whole.table, ints(now), starts_of(rows))
    a = whole.everything()
    b = W.kv4_read(other, whole.table, whole.len, starts_of(lengths), rows=sum(lengths))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    W.device_check()


@pytest.mark.parametrize("rows", [[3, 1, 2], [100, 70, 0], [130, 200, 65]])
def test_reading_rows_from_anywhere_and_without_tokens(W, rows):
    """The last rows of each sequence, which may be more than it holds: those read as zeros."""
    lengths = [99, 130, 64]
    b = Batch(W, lengths, 2, 128, seed=7)
    n = (sum(rows) + 2) * 2 * 128
    flat = torch.full((2 * (n + 2 * GUARD),), 7.0, dtype=torch.bfloat16, device="cuda")
    for shift in (0, 1):  # 16-byte aligned or not
        k, v = (flat[i * (n + 2 * GUARD) + GUARD + shift:][:n].view(-1, 2, 128) for i in range(2))
        W.kv4_read(b.cache, b.table, b.len, starts_of(rows), k=k, v=v)
        at = 0
        for i, r in enumerate(rows):
            for got, held in ((k, b.ks[i]), (v, b.vs[i])):
                want = np.concatenate([np.zeros((max(0, r - lengths[i]), 2, 128)), held[max(0, lengths[i] - r):]])
                same_values(bits(got[at:at + r]), want)
            at += r
        k[:at].fill_(7.0), v[:at].fill_(7.0)
        assert (flat == 7.0).all()
    W.device_check()


@pytest.mark.parametrize("D", [64, 128, 256])
def test_append_of_strided_and_unaligned_rows(W, D):
    rng = np.random.default_rng(2)
    T, H = 37, 3
    b = Batch(W, [0], H, D, width=2)
    lengths = ints([T])
    whole = dev16(draw((T, 2 * H + 1, D), rng))
    cases = [(whole[:, 1:H + 1], whole[:, H + 1:]),                       # heads of one tensor
             (whole[:, 0:2 * H:2], whole[:, 1:2 * H + 1:2]),              # every other head
             (whole.transpose(0, 1).contiguous().transpose(0, 1)[:, :H],) * 2]  # heads outermost
    odd = torch.empty(T * H * D + 1, dtype=torch.bfloat16, device="cuda")[1:].view(T, H, D)
    odd.copy_(whole[:, :H])
    cases.append((odd, whole[:, :H]))                                     # a base that is 2-byte aligned
    cases.append((whole[:1, :H].expand(T, H, D), whole[:, :1].expand(T, H, D)))  # broadcast rows and heads
    for k, v in cases:
        W.kv4_append(b.cache, k, v, b.table, lengths, ints([0, T]))
        got = W.kv4_read(b.cache, b.table, lengths, ints([0, T]), rows=T)
        same_values(bits(got[0]), K.held(bits(k)))
        same_values(bits(got[1]), K.held(bits(v)))
    W.device_check()


def test_every_bf16_magnitude_as_a_groups_largest(W):
    tops = np.arange(1, 0x7F80, dtype=np.uint16)
    rng = np.random.default_rng(1)
    scale = f64(bf16(f64(tops) / 7.0))
    rows = np.zeros((len(tops), 32), np.uint16)
    for i in range(1, 32):
        v = bf16(scale * (rng.integers(-13, 14, len(tops)) / 2.0)).astype(np.int64) + rng.integers(-1, 2, len(tops))
        rows[:, i] = (np.clip(v & 0x7FFF, 0, tops) | (v & 0x8000)).astype(np.uint16)
    rows[:, 0] = tops
    rows = np.concatenate([rows, np.zeros((-len(rows) % 4, 32), np.uint16)]).reshape(-1, 1, 128)
    b = Batch(W, [len(rows)], 1, 128, k=rows, v=rows[::-1].copy())
    k, v = b.everything()
    same_values(bits(k), K.held(b.k))
    same_values(bits(v), K.held(b.v))


def test_non_finite_groups_become_nan_and_no_others(W):
    k = np.full((3, 1, 64), 0x3F80, np.uint16)
    k[0, 0, 3], k[1, 0, 40], k[2, 0, 0] = 0x7F80, 0x7FC1, 0xFF80
    b = Batch(W, [3], 1, 64, k=k, v=k)
    for t in b.everything():
        bad = np.isnan(f64(bits(t)))
        assert bad[0, 0, :32].all() and not bad[0, 0, 32:].any() and bad[1, 0, 32:].all() and not bad[1, 0, :32].any()
        assert bad[2, 0, :32].all()


def test_rows_of_no_sequence_and_guards_are_left_alone(W):
    """Outputs between guards; rows behind the last sequence, and pages of nobody, keep what they held."""
    b = Batch(W, [5, 0, 66], 2, 64, spare=8)
    before = W.kv4_read(b.cache, ints(np.arange(b.pages)[None]), ints([b.pages * 64]), ints([0, b.pages * 64]),
                        rows=b.pages * 64)
    starts = ints([0, 2, 3, 6])  # the second sequence has a row and no tokens; rows 6 to 8 are nobody's
    n = 9 * 2 * 64
    flat = torch.full((2 * (n + 2 * GUARD),), 7.0, dtype=torch.bfloat16, device="cuda")
    k, v = (flat[i * (n + 2 * GUARD) + GUARD:][:n].view(9, 2, 64) for i in range(2))
    W.kv4_read(b.cache, b.table, b.len, starts, k=k, v=v)
    want = np.concatenate([K.held(b.k)[3:5], np.zeros((1, 2, 64)), K.held(b.k)[-3:]])
    same_values(bits(k[:6]), want)
    k.fill_(7.0), v[:6].fill_(7.0)
    assert (flat == 7.0).all()
    junk = dev16(draw((9, 2, 64), np.random.default_rng(1)))
    W.kv4_append(b.cache, junk, junk, b.table, b.len, starts)
    after = W.kv4_read(b.cache, ints(np.arange(b.pages)[None]), ints([b.pages * 64]), ints([0, b.pages * 64]),
                       rows=b.pages * 64)
    changed = (bits(before[0]) != bits(after[0])).any((1, 2)) | (bits(before[1]) != bits(after[1])).any((1, 2))
    place = [b.table_np[0, 0] * 64 + i for i in (3, 4)] + [b.table_np[2, 0] * 64 + 63] + [
        b.table_np[2, 1] * 64 + i for i in (0, 1)]
    assert set(np.nonzero(changed)[0]) <= set(place) and changed[place].all()
    W.device_check()


# ---------------------------------------------------------------------------
# Attention.
# ---------------------------------------------------------------------------
def attend_matches(W, b, q, rows, scale=None, window=0, starts=True, strided=False, extra=0):
    """One call with every output against the definition; returns (out, lse, mass)."""
    T, Hq, D = q.shape
    B, H, scale_v = len(b.lengths), b.H, D ** -0.5 if scale is None else scale
    qd = dev16(q)
    if strided:
        wide = torch.zeros(T, Hq + 2, D + 8, dtype=torch.bfloat16, device="cuda")
        wide[:, 1:-1, 4:-4] = qd
        qd = wide[:, 1:-1, 4:-4]
    out = torch.full((T * Hq * D + 2 * GUARD,), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((T * Hq + 2 * GUARD,), 7.0, device="cuda")
    mass = torch.full((B * H * b.width * 64 + 2 * GUARD,), 7.0, device="cuda")
    o, l = out[GUARD:-GUARD].view(T, Hq, D), lse[GUARD:-GUARD].view(T, Hq)
    m = mass[GUARD:-GUARD].view(B, H, -1)
    m.copy_(torch.rand(m.shape, generator=torch.Generator().manual_seed(3)))
    m0 = m.cpu().numpy().astype(np.float64)
    got = W.kv4_attend(b.cache, qd, b.table, b.len, starts_of(rows) if starts else None, scale=scale, window=window,
                       out=o, lse=l, mass=m)
    assert got.data_ptr() == o.data_ptr()
    on, ln, mn = f64(bits(o)), l.cpu().numpy().astype(np.float64), m.cpu().numpy().astype(np.float64)
    at = 0
    for i, r in enumerate(rows):
        wo, wl, wm, to, tl, tm = K.attend(f64(q[at:at + r]), b.ks[i], b.vs[i], scale_v, window)
        assert (np.abs(on[at:at + r] - wo) <= to).all(), (i, np.abs(on[at:at + r] - wo).max())
        empty = np.isneginf(wl)
        assert np.array_equal(np.isneginf(ln[at:at + r]), empty)
        assert (np.abs(ln[at:at + r][~empty] - wl[~empty]) <= tl[~empty]).all(), i
        n = b.lengths[i]
        err = np.abs(mn[i, :, :n] - m0[i, :, :n] - wm)
        assert (err <= tm + 4 * K.EPS * mn[i, :, :n]).all(), (i, err.max())
        assert np.array_equal(mn[i, :, n:], m0[i, :, n:])  # places without a token
        at += r
    assert (o[at:] == 7.0).all() and (l[at:] == 7.0).all()  # rows of no sequence
    o.fill_(7.0), l.fill_(7.0), m.fill_(7.0)
    assert (out == 7.0).all() and (lse == 7.0).all() and (mass == 7.0).all()
    return on, ln, mn


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("share", [1, 2, 7, 8, 9, 16, 40])
def test_attention_of_single_tokens(W, D, share):
    lengths = [1, 64, 0, 65, 63, 200, 2]
    b = Batch(W, lengths, 2, D, seed=share)
    q = draw((7, 2 * share, D), np.random.default_rng(share), 1.5)
    attend_matches(W, b, q, [1] * 7, starts=False)
    W.device_check()


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("share", [1, 4, 5])
@pytest.mark.parametrize("window", [0, 1, 3, 64, 100])
def test_attention_of_several_tokens(W, D, share, window):
    """Ragged rows: none, one, more than the sequence holds, a whole short prompt; a causal order among them."""
    lengths, rows = [130, 5, 65, 3, 0, 77], [4, 5, 0, 6, 2, 1]
    b = Batch(W, lengths, 3, D, seed=share + window)
    q = draw((sum(rows) + 3, 3 * share, D), np.random.default_rng(window), 1.5)
    attend_matches(W, b, q, rows, window=window, strided=share == 5)
    W.device_check()


@pytest.mark.parametrize("D,share,n", [(128, 4, 5000), (64, 8, 3333), (256, 3, 2100), (128, 16, 2500)])
def test_attention_over_long_sequences(W, D, share, n):
    b = Batch(W, [n, 17, n // 3], 2, D, seed=n)
    q = draw((3, 2 * share, D), np.random.default_rng(n), 2.0)
    attend_matches(W, b, q, [1, 1, 1], starts=False)
    attend_matches(W, b, q, [1, 1, 1], window=n // 2 + 5)
    W.device_check()


@pytest.mark.parametrize("D,share,window", [(64, 3, 0), (128, 1, 0), (128, 4, 100), (256, 2, 0)])
def test_attention_of_whole_prompts(W, D, share, window):
    """Every row of its prompt: many tiles of rows, each of which sees more pages than the one before."""
    lengths = [333, 1, 150]
    b = Batch(W, lengths, 2, D, seed=D)
    q = draw((sum(lengths), 2 * share, D), np.random.default_rng(D + share), 1.5)
    attend_matches(W, b, q, lengths, window=window)
    W.device_check()


@pytest.mark.parametrize("D,share", [(64, 8), (128, 4), (128, 12), (256, 1)])
@pytest.mark.parametrize("B,width", [(1, 33), (2, 500), (3, 90), (9, 60), (20, 49), (40, 17), (76, 5), (77, 5),
                                     (2, 1100), (20, 160), (100, 9)])
def test_attention_by_blocks_and_clusters_of_any_size(W, D, share, B, width):
    """Batches that leave a tile one to sixteen blocks, and those whose tables are too wide for that."""
    rng = np.random.default_rng(B)
    lengths = [int(n) for n in rng.integers(0, 64 * min(width, 12) + 1, B)]
    lengths[-1] = min(64 * width, 1500)
    b = Batch(W, lengths, 2, D, seed=B, width=width)
    q = draw((B, 2 * share, D), rng, 1.5)
    attend_matches(W, b, q, [1] * B, starts=False)
    attend_matches(W, b, q, [1] * B, starts=False, window=100)
    W.device_check()


@pytest.mark.parametrize("scale", [0.0, -0.25, 1e-6, 3.0])
def test_attention_with_other_scales(W, scale):
    b = Batch(W, [300, 64], 2, 128, seed=4)
    attend_matches(W, b, draw((2, 8, 128), np.random.default_rng(8)), [1, 1], scale=scale)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("kq,kk,kv", [(2.0 ** -60, 2.0 ** 62, 1.0), (2.0 ** 50, 2.0 ** -52, 2.0 ** 100),
                                      (1.0, 1.0, 2.0 ** -120), (2.0 ** -110, 1.0, 2.0 ** 120), (0.0, 1.0, 1.0)])
def test_attention_keeps_its_bits_at_every_magnitude(W, D, kq, kk, kv):
    rng = np.random.default_rng(3)
    k, v = bf16(rng.standard_normal((190, 2, D)) * kk), bf16(rng.standard_normal((190, 2, D)) * kv)
    b = Batch(W, [150, 40], 2, D, k=k, v=v)
    q = bf16(rng.standard_normal((2, 6, D)) * kq)
    attend_matches(W, b, q, [1, 1], starts=False)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("size", [2.0 ** 21, 2.0 ** 24, 2.0 ** 33, 2.0 ** 60, 2.0 ** 103])  # |q k| sums to less than 2^112
@pytest.mark.parametrize("n", [150, 2000])  # joined in a cluster's shared memory, and cut anywhere
def test_scores_far_apart_and_from_zero_choose_one_token(W, D, size, n):
    """Scores that fp32 has whole steps between; the largest is alone by more than its error, so its token's value is
    the result, its score the log-sum-exp and its mass 1, also as values that grow move the sums' power of two."""
    rng = np.random.default_rng(n)
    k = rng.standard_normal((n, 2, D)) * size
    v = rng.standard_normal((n, 2, D)) * 2.0 ** np.repeat(rng.integers(-40, 40, (n + 63) // 64), 64)[:n, None, None]
    b = Batch(W, [n], 2, D, k=bf16(k), v=bf16(v), width=3 if n < 500 else 800)
    q = bf16(rng.standard_normal((1, 6, D)))
    lse, mass = torch.empty(1, 6, device="cuda"), torch.zeros(1, 2, b.width * 64, device="cuda")
    out = f64(bits(W.kv4_attend(b.cache, dev16(q), b.table, b.len, scale=1.0, lse=lse, mass=mass)))
    weight = np.zeros((2, n))
    for h in range(6):
        z = b.ks[0][:, h // 3] @ f64(q[0, h])
        mag = np.abs(b.ks[0][:, h // 3]) @ np.abs(f64(q[0, h]))
        top, second = np.argsort(z)[:-3:-1]
        off = K.EPS * (D / 4 + 8) * mag.max()
        if z[top] - z[second] < 2 * off + 40:  # less, and what of the other is left shows
            continue
        want = b.vs[0][top, h // 3]
        assert (np.abs(out[0, h] - want) <= (2.0 ** -8 + 2.0 ** -10) * np.abs(want)).all(), h
        assert abs(float(lse[0, h]) - z[top]) <= off + 4 * K.EPS * abs(z[top])
        weight[h // 3, top] += 1
    got = mass[0, :, :n].cpu().numpy().astype(np.float64)
    assert np.isfinite(got).all() and (got >= weight * (1 - 2.0 ** -9)).all()
    assert weight.sum() >= 3


def test_attention_to_one_token_among_many(W):
    """A token whose score stands out, anywhere, also after pages of others; values of very different scales."""
    rng = np.random.default_rng(6)
    n = 500
    for at in (0, 63, 64, 300, 499):
        k, v = rng.standard_normal((n, 1, 128)), rng.standard_normal((n, 1, 128))
        v *= 2.0 ** rng.integers(-12, 12, (n, 1, 1))
        q = rng.standard_normal((1, 4, 128))
        k[at] = 3 * q[0, 1]
        b = Batch(W, [n], 1, 128, k=bf16(k), v=bf16(v))
        attend_matches(W, b, bf16(q), [1])


@pytest.mark.parametrize("D", [64, 128, 256])
def test_infinities_and_nan_where_a_row_does_not_look_change_nothing(W, D):
    rng = np.random.default_rng(9)
    n, rows, window = 150, 3, 70
    k, v = draw((n, 2, D), rng), draw((n, 2, D), rng)
    b = Batch(W, [n], 2, D, k=k, v=v)
    q = dev16(draw((rows, 4, D), rng))
    call = lambda: (lambda l: (bits(W.kv4_attend(b.cache, q, b.table, b.len, ints([0, rows]), window=window, lse=l)),
                               l.cpu().numpy()))(torch.empty(rows, 4, device="cuda"))
    out, lse = call()
    bad = dev16(np.full((1, 2, D), 0x7FC0, np.uint16))
    # outside every window; then the first place behind the sequence
    for at in (n - rows - window, n):
        W.kv4_append(b.cache, bad, bad, b.table, ints([at + 1]))
        got, got_lse = call()
        assert np.array_equal(got, out) and np.array_equal(got_lse, lse)
    # the last token: seen by the last row alone, in one head
    half = bad.clone()
    half[:, 1] = 1.0
    W.kv4_append(b.cache, dev16(k[-1:]), half, b.table, b.len)
    got, got_lse = call()
    assert np.array_equal(got[:2], out[:2]) and np.array_equal(got_lse, lse)
    assert np.isnan(f64(got[2, :2])).all() and np.isfinite(f64(got[2, 2:])).all()
    W.kv4_append(b.cache, half, dev16(v[-1:]), b.table, b.len)
    got, got_lse = call()
    assert np.array_equal(got[:2], out[:2]) and np.array_equal(got_lse[:2], lse[:2])
    assert np.isnan(f64(got[2, :2])).all() and np.isnan(got_lse[2, :2]).all() and np.isfinite(got_lse[2, 2:]).all()


def test_a_group_of_nan_values_stays_in_its_columns(W):
    rng = np.random.default_rng(10)
    k, v = draw((80, 1, 128), rng), draw((80, 1, 128), rng)
    v[70, 0, 40] = 0x7F80
    b = Batch(W, [80], 1, 128, k=k, v=v)
    q = draw((1, 4, 128), rng)
    out = f64(bits(W.kv4_attend(b.cache, dev16(q), b.table, b.len)))
    assert np.isnan(out[..., 32:64]).all()
    keep = np.r_[0:32, 64:128]
    b.vs[0][:, :, 32:64] = 0.0
    want, _, _, tol, _, _ = K.attend(f64(q), b.ks[0], b.vs[0], 128 ** -0.5)
    assert (np.abs(out - want)[..., keep] <= tol[..., keep]).all()


def test_queries_that_are_not_finite(W):
    rng = np.random.default_rng(11)
    b = Batch(W, [100], 1, 64, seed=2)
    q = draw((1, 9, 64), rng)
    want = bits(W.kv4_attend(b.cache, dev16(q), b.table, b.len))
    q[0, 2, 5], q[0, 8, 0] = 0x7FC0, 0x7F80
    got = bits(W.kv4_attend(b.cache, dev16(q), b.table, b.len))
    assert np.isnan(f64(got[0, [2, 8]])).all()
    rest = [0, 1, 3, 4, 5, 6, 7]
    assert np.array_equal(got[0, rest], want[0, rest])


@pytest.mark.parametrize("D,share", [(64, 16), (128, 8)])
def test_weights_do_not_depend_on_how_they_are_found(W, D, share):
    """From kept scores, from the keys again (too many scores to keep; rows given by starts), by a cluster."""
    rng = np.random.default_rng(21)
    H, width, B = 8, 1300, 16 if share == 8 else 8
    n = 64 * width - 5
    b = Batch(W, [3000], H, D, seed=2)
    pages = b.table_np[0, :46]  # every sequence reads these again and again
    table = ints(np.resize(pages, (B, width)))
    lengths = ints([n, 0, 1, 700] + [100 * i for i in range(4, B)])
    q = dev16(draw((B, H * share, D), rng, 1.5))

    def weights(rows, wide=width, starts=None):
        mass = torch.zeros(rows, H, wide * 64, device="cuda")
        W.kv4_attend(b.cache, q[:rows], table[:rows, :wide].contiguous(), lengths[:rows].clamp(max=64 * wide), starts,
                     mass=mass)
        return mass.double().cpu()

    again, kept, started = weights(B), weights(4), weights(B, starts=ints(range(B + 1)))
    for got in (kept, started[:4]):
        # scores and log-sum-exps of at most 32 are rounded at other places, 2^-19 each; sums of exponentials run in
        # parts of at most 48 tokens a lane and 304 parts, 352 EPS; both in either call: below 2^-14
        assert ((got - again[:4]).abs() <= 2 ** -14 * again[:4] + 1e-30).all()
    few = weights(B, wide=30)[4:]
    assert ((few - again[4:, :, :30 * 64]).abs() <= 2 ** -14 * few + 1e-30).all()
    assert (again[0].sum(1) - share).abs().max() <= 2 ** -14 * share and (again[1] == 0).all()
    W.device_check()


def test_sequences_that_share_pages(W):
    """A common prefix is held once; sequences go on in pages of their own."""
    b = Batch(W, [128, 0, 0], 2, 128, width=4)
    table = b.table_np.copy()
    table[1:, :2] = table[0, :2]
    b.table, b.table_np = ints(table), table
    rng = np.random.default_rng(12)
    k, v = draw((9, 2, 128), rng), draw((9, 2, 128), rng)
    b.lengths, b.len = [128, 131, 134], ints([128, 131, 134])
    W.kv4_append(b.cache, dev16(k), dev16(v), b.table, b.len, ints([0, 0, 3, 9]))
    b.ks = [b.ks[0], np.concatenate([b.ks[0], K.held(k[:3])]), np.concatenate([b.ks[0], K.held(k[3:])])]
    b.vs = [b.vs[0], np.concatenate([b.vs[0], K.held(v[:3])]), np.concatenate([b.vs[0], K.held(v[3:])])]
    attend_matches(W, b, draw((10, 8, 128), rng), [1, 3, 6])


def test_a_page_named_twice_by_one_sequence(W):
    b = Batch(W, [64], 1, 64, width=3)
    b.table[0, 1] = b.table[0, 0]
    b.lengths, b.len = [128], ints([128])
    b.ks, b.vs = [np.concatenate([b.ks[0]] * 2)], [np.concatenate([b.vs[0]] * 2)]
    attend_matches(W, b, draw((1, 4, 64), np.random.default_rng(1)), [1])


@pytest.mark.parametrize("lengths,rows", [([90], [1]), ([9000, 200], [1, 1]), ([3000, 70], [3, 2])])
def test_unaligned_outputs(W, lengths, rows):
    """out and q from 2-byte boundaries: the same bits, by each kernel."""
    b = Batch(W, lengths, 2, 128, seed=8)
    q = dev16(draw((sum(rows), 8, 128), np.random.default_rng(1)))
    want = W.kv4_attend(b.cache, q, b.table, b.len, starts_of(rows))
    for off in (1, 2, 3, 5):
        flat = torch.full((2 * q.numel() + 64,), 7.0, dtype=torch.bfloat16, device="cuda")
        odd_q, out = flat[off:off + q.numel()].view(q.shape), flat[q.numel() + 32 + off:][:q.numel()].view(q.shape)
        odd_q.copy_(q)
        W.kv4_attend(b.cache, odd_q, b.table, b.len, starts_of(rows), out=out)
        assert torch.equal(out, want)
        out.fill_(7.0), odd_q.fill_(7.0)
        assert (flat == 7.0).all()
    k = torch.empty(sum(lengths) * 256 + 1, dtype=torch.bfloat16, device="cuda")[1:].view(-1, 2, 128)
    W.kv4_read(b.cache, b.table, b.len, starts_of(lengths), k=k, v=torch.empty_like(k))
    same_values(bits(k), K.held(b.k))
    W.device_check()


def test_no_rows_and_no_sequences(W):
    b = Batch(W, [10], 2, 64)
    none = torch.empty(0, 4, 64, dtype=torch.bfloat16, device="cuda")
    assert W.kv4_attend(b.cache, none, b.table, b.len, ints([0, 0])).shape == (0, 4, 64)
    assert W.kv4_attend(b.cache, none, b.table[:0], b.len[:0]).shape == (0, 4, 64)
    W.kv4_append(b.cache, none[:, :2], none[:, :2], b.table, b.len, ints([0, 0]))
    assert W.kv4_read(b.cache, b.table[:0], b.len[:0])[0].shape == (0, 2, 64)
    W.device_check()


def test_many_sequences(W):
    """More sequences than a block has threads, most of them short; calls repeat bit for bit."""
    rng = np.random.default_rng(13)
    lengths = [int(n) for n in rng.integers(0, 40, 700)]
    lengths[123], lengths[699] = 1000, 500
    b = Batch(W, lengths, 1, 64, seed=1)
    rows = [int(r) for r in rng.integers(0, 4, 700)]
    q = draw((sum(rows), 3, 64), rng)
    first = attend_matches(W, b, q, rows)
    again = attend_matches(W, b, q, rows)
    assert all(np.array_equal(x, y) for x, y in zip(first, again))
    W.device_check()


# ---------------------------------------------------------------------------
# Bad pages, lengths and arguments.
# ---------------------------------------------------------------------------
def reported(W):
    with pytest.raises(W.WcompError) as e:
        W.device_check()
    assert e.value.status == W.EBOUNDS
    W.device_check()  # cleared


def test_pages_and_lengths_out_of_range_are_skipped_and_reported(W):
    rng = np.random.default_rng(14)
    b = Batch(W, [200, 100], 2, 64, width=4)
    q = dev16(draw((2, 4, 64), rng))
    want = W.kv4_attend(b.cache, q, b.table, b.len)
    W.device_check()
    for page in (-1, b.pages, 2 ** 31 - 1, -2 ** 31):
        table = b.table.clone()
        table[0, 1] = page
        got = W.kv4_attend(b.cache, q, table, b.len)
        reported(W)
        assert torch.equal(got[1], want[1])
        # as if tokens 64 to 127 were not there
        keep = np.r_[0:64, 128:200]
        o, _, _, tol, _, _ = K.attend(f64(bits(q[:1])), b.ks[0][keep], b.vs[0][keep], 64 ** -0.5)
        assert (np.abs(f64(bits(got[:1])) - o) <= tol).all()
        k, v = W.kv4_read(b.cache, table, b.len, ints([0, 200, 200]), rows=200)
        reported(W)
        assert (k[64:128] == 0).all() and (v[64:128] == 0).all()
        same_values(bits(k)[keep], b.ks[0][keep])
        W.kv4_append(b.cache, k, v, table, b.len, ints([0, 200, 200]))
        reported(W)
        mass = torch.zeros(2, 2, 256, device="cuda")
        W.kv4_attend(b.cache, q, table, b.len, mass=mass)
        reported(W)
        assert (mass[0, :, 64:128] == 0).all() and (mass[0, :, :64] > 0).all()
    # the last append wrote what was read: everything but the skipped page is as it was
    long = W.kv4_attend(b.cache, q[:1], b.table[1:, :2].contiguous(), ints([129]))  # more than two pages hold
    reported(W)
    full = W.kv4_attend(b.cache, q[:1], b.table[1:, :2].contiguous(), ints([128]))
    assert torch.equal(long, full)
    assert (W.kv4_attend(b.cache, q, b.table, ints([-5, 0])) == 0).all()
    W.device_check()


def test_starts_out_of_range_reach_nothing_outside(W):
    """Rows are those of the call whatever starts say."""
    b = Batch(W, [70, 30], 1, 64)
    q = torch.full((4 + 2 * 64, 2, 64), 1.0, dtype=torch.bfloat16, device="cuda")
    for s in ([0, 2, 1000], [5, 2, 0], [-7, 2, 4], [0, 1000, 4], [0, 2 ** 31 - 1, 2 ** 31 - 1], [-2 ** 31, -5, 3]):
        out = torch.full_like(q, 7.0)
        lse = torch.full((4 + 128, 2), 7.0, device="cuda")
        mass = torch.zeros(2, 1, b.width * 64, device="cuda")
        W.kv4_attend(b.cache, q[64:68], b.table, b.len, ints(s), out=out[64:68], lse=lse[64:68], mass=mass)
        k = torch.full((4 + 128, 1, 64), 7.0, dtype=torch.bfloat16, device="cuda")
        W.kv4_read(b.cache, b.table, b.len, ints(s), k=k[64:68], v=k[64:68].clone())
        for t in (out, lse, k):
            assert (t[:64] == 7.0).all() and (t[68:] == 7.0).all()
    torch.cuda.synchronize()
    try:
        W.device_check()
    except W.WcompError as e:
        assert e.status == W.EBOUNDS


def test_the_abi_refuses_bad_arguments_for_a_real_cache(W):
    L = W.lib()
    b = Batch(W, [10, 10], 2, 64, width=2)
    h = b.cache.handle
    s = W.Kv4Seqs(b.table.data_ptr(), b.len.data_ptr(), None, 2, 2)
    p = torch.zeros(4, 2, 64, dtype=torch.bfloat16, device="cuda").data_ptr()
    r = ctypes.byref

    def bad(**kw):
        x = W.Kv4Seqs(s.d_table, s.d_lengths, s.d_starts, s.B, s.width)
        for n, v in kw.items():
            setattr(x, n, v)
        return x

    for x in (bad(d_table=None), bad(d_lengths=None), bad(d_table=s.d_table + 1), bad(d_lengths=s.d_lengths + 2),
              bad(d_starts=s.d_table + 1), bad(B=-1), bad(width=0), bad(B=3)):
        assert L.wcomp_kv4_append(h, r(x), p, 128, 64, p, 128, 64, 2, None) == W.EINVAL
        assert L.wcomp_kv4_read(h, r(x), p, p, 2, None) == W.EINVAL
        assert L.wcomp_kv4_attend(h, r(W.Kv4AttendArgs(x, p, 128, 64, p, None, None, 2, 2, 0, 1.0)), None) == W.EINVAL
    assert L.wcomp_kv4_append(h, r(s), None, 128, 64, p, 128, 64, 2, None) == W.EINVAL
    assert L.wcomp_kv4_append(h, r(s), p, 128, 64, None, 128, 64, 2, None) == W.EINVAL
    assert L.wcomp_kv4_append(h, r(s), p, -128, 64, p, 128, 64, 2, None) == W.EINVAL
    assert L.wcomp_kv4_append(h, r(s), p, 128, 64, p, 128, 64, -2, None) == W.EINVAL
    assert L.wcomp_kv4_append(h, None, p, 128, 64, p, 128, 64, 2, None) == W.EINVAL
    assert L.wcomp_kv4_read(h, r(s), None, p, 2, None) == W.EINVAL
    assert L.wcomp_kv4_read(h, r(bad(width=1 << 26)), p, p, 2, None) == W.EUNSUPPORTED
    f0 = torch.zeros(8, device="cuda").data_ptr()
    ok = (s, p, 128, 64, p + 512, None, None, 2, 2, 0, 1.0)
    for i, v in ((1, None), (1, p + 1), (4, p), (4, p + 1), (5, f0 + 2), (6, f0 + 2), (2, -1), (3, -1), (4, None), (7, -1), (8, 3), (8, 0), (9, -1), (10, float("nan")),
                 (10, float("inf"))):
        a = list(ok)
        a[i] = v
        assert L.wcomp_kv4_attend(h, r(W.Kv4AttendArgs(*a)), None) == W.EINVAL, (i, v)
    f = torch.zeros(2, 2, 128, device="cuda").data_ptr()
    g = torch.zeros(2, 2, 128, device="cuda").data_ptr()
    out = b.table.clone()
    ev = (s.d_table, s.d_lengths, f, out.data_ptr(), b.len.clone().data_ptr(), g, None, 2, 2, 2, 4, 1)
    for i, v in ((0, None), (1, None), (2, None), (3, None), (3, s.d_table), (4, None), (4, s.d_lengths), (5, None), (5, f),
                 (0, s.d_table + 2), (2, f + 2), (6, f + 1), (7, -1),
                 (8, 0), (9, 0), (10, 0), (10, 129), (11, -1), (11, 5)):
        a = list(ev)
        a[i] = v
        assert L.wcomp_kv4_evict(h, r(W.Kv4EvictArgs(*a)), None) == W.EINVAL, (i, v)
    info = b.cache.info()
    assert info == {"pages": b.pages, "heads": 2, "dim": 64, "bytes": b.pages * 2 * 72 * 64}
    W.device_check()


# ---------------------------------------------------------------------------
# Eviction.
# ---------------------------------------------------------------------------
def evict_matches(W, b, mass, keep, recent, outputs=True):
    B, H = len(b.lengths), b.H
    wide = -(-keep // 64) + 1
    old = b.pages
    bigger = W.kv4_create(old + B * wide, H, b.D)
    W.kv4_append(bigger, dev16(b.k), dev16(b.v), b.table, b.len, starts_of(b.lengths))
    rng = np.random.default_rng(keep)
    table_out = ints(old + rng.permutation(B * wide).reshape(B, wide))
    flat = torch.full((B * H * keep + 2 * GUARD,), 99, dtype=torch.int32, device="cuda")
    kept = flat[GUARD:-GUARD].view(B, H, keep)
    before = W.kv4_read(bigger, b.table, b.len, starts_of(b.lengths), rows=sum(b.lengths))
    lengths, mass_out = W.kv4_evict(bigger, b.table, b.len, torch.from_numpy(mass).cuda(), keep, recent, table_out,
                                    kept=kept if outputs else None)
    assert lengths.tolist() == [min(n, keep) for n in b.lengths]
    m = lengths.tolist()
    k, v = (bits(t) for t in W.kv4_read(bigger, table_out, lengths, starts_of(m), rows=sum(m)))
    after = W.kv4_read(bigger, b.table, b.len, starts_of(b.lengths), rows=sum(b.lengths))
    assert torch.equal(before[0], after[0]) and torch.equal(before[1], after[1])
    kn, mn = kept.cpu().numpy(), mass_out.cpu().numpy()
    at = 0
    for i, n in enumerate(b.lengths):
        for h in range(H):
            want = K.evict(mass[i, h], n, keep, recent)
            if outputs:
                assert np.array_equal(kn[i, h, :m[i]], want) and (kn[i, h, m[i]:] == -1).all()
            assert np.array_equal(mn[i, h, :m[i]], mass[i, h, want], equal_nan=True) and (mn[i, h, m[i]:] == 0).all()
            same_values(k[at:at + m[i], h], b.ks[i][want, h])
            same_values(v[at:at + m[i], h], b.vs[i][want, h])
        at += m[i]
    kept.fill_(99)
    assert (flat == 99).all()
    W.device_check()


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("keep,recent", [(1, 0), (1, 1), (64, 10), (65, 0), (100, 100), (130, 33), (400, 20)])
def test_eviction_is_the_definition(W, D, keep, recent):
    b = Batch(W, [300, 0, 1, 64, 65, 130, 129, 1100], 2, D, seed=keep)
    rng = np.random.default_rng(recent)
    mass = (rng.random((8, 2, b.width * 64)) ** 4).astype(np.float32)
    evict_matches(W, b, mass, keep, recent)


@pytest.mark.parametrize("keep,recent", [(7, 2), (150, 0), (1500, 1)])
def test_eviction_with_ties_and_odd_masses(W, keep, recent):
    """Equal masses, zeros of both signs, negative ones, infinities and NaN: the lowest positions win."""
    b = Batch(W, [2500, 700, 160], 2, 64, seed=3)
    rng = np.random.default_rng(7)
    mass = rng.choice(np.array([0.0, -0.0, 1.0, 1.0, -1.0, np.inf, -np.inf, np.nan, 1e-45, -1e-45], np.float32),
                      (3, 2, b.width * 64))
    mass[0, 1] = 0.0
    evict_matches(W, b, mass, keep, recent)
    evict_matches(W, b, mass, keep, recent, outputs=False)


def test_eviction_goes_on_from_an_eviction(W):
    """A cache is kept at a size: evicted, grown, attended to and evicted again."""
    rng = np.random.default_rng(15)
    n, keep, recent, H, D = 200, 96, 16, 2, 128
    b = Batch(W, [n, n - 50], H, D, width=4, spare=12)
    free = [p for p in range(b.pages) if p not in set(b.table_np.flatten())]
    table2 = ints(np.array(free[:8]).reshape(2, 4))
    q = draw((2, 8, D), rng, 2.0)
    _, _, mass = attend_matches(W, b, q, [1, 1])
    m = torch.from_numpy(mass.astype(np.float32)).cuda()
    kept = torch.empty(2, H, keep, dtype=torch.int32, device="cuda")
    wide = torch.empty(2, H, 4 * 64, device="cuda")
    lengths, m2 = W.kv4_evict(b.cache, b.table, b.len, m, keep, recent, table2, kept=kept, mass_out=wide)
    assert m2.data_ptr() == wide.data_ptr()
    kn = kept.cpu().numpy()
    b.ks = [np.stack([b.ks[i][kn[i, h], h] for h in range(H)], 1) for i in range(2)]
    b.vs = [np.stack([b.vs[i][kn[i, h], h] for h in range(H)], 1) for i in range(2)]
    k, v = draw((2, H, D), rng), draw((2, H, D), rng)
    b.table, b.width, b.lengths, b.len = table2, 4, [keep + 1, keep + 1], lengths + 1
    W.kv4_append(b.cache, dev16(k), dev16(v), b.table, b.len)
    b.ks = [np.concatenate([b.ks[i], K.held(k[i:i + 1])]) for i in range(2)]
    b.vs = [np.concatenate([b.vs[i], K.held(v[i:i + 1])]) for i in range(2)]
    attend_matches(W, b, draw((2, 8, D), rng, 2.0), [1, 1], starts=False)
    lengths, m3 = W.kv4_evict(b.cache, b.table, b.len, m2, 64, 8, ints(np.array(free[8:12]).reshape(2, 2)), kept=None)
    assert lengths.tolist() == [64, 64] and m3.shape == (2, H, 128)
    W.device_check()


def test_eviction_into_bad_pages_is_reported(W):
    b = Batch(W, [100], 1, 64, width=2, spare=4)
    free = [p for p in range(b.pages) if p not in set(b.table_np.flatten())]
    mass = torch.rand(1, 1, 128, device="cuda")
    W.kv4_evict(b.cache, b.table, b.len, mass, 70, 5, ints([[free[0], b.pages]]))
    reported(W)
    same = b.everything()
    same_values(bits(same[0]), K.held(b.k))


def test_a_cache_that_finds_no_memory(W):
    """2^43 bytes are refused, and the next calls are as before."""
    b = Batch(W, [70], 2, 64, seed=1)
    q = dev16(draw((1, 4, 64), np.random.default_rng(1)))
    want = W.kv4_attend(b.cache, q, b.table, b.len)
    h = ctypes.c_void_p(1)
    assert W.lib().wcomp_kv4_create((1 << 31) // 2 - 1, 1, 256, None, ctypes.byref(h)) == W.ENOMEM and not h.value
    assert torch.equal(W.kv4_attend(b.cache, q, b.table, b.len), want)
    W.device_check()


def test_memory_comes_back(W):
    """Caches made and dropped, calls with workspaces: the device's free memory does not shrink."""
    def work():
        b = Batch(W, [3000, 10], 4, 128, seed=1)
        q = dev16(draw((2, 16, 128), np.random.default_rng(1)))
        mass = torch.zeros(2, 4, b.width * 64, device="cuda")
        for _ in range(5):
            W.kv4_attend(b.cache, q, b.table, b.len, mass=mass)
            W.kv4_evict(b.cache, b.table, b.len, mass, 10, 2, ints([[b.pages - 1], [b.pages - 2]]))
        b.cache.free()
        torch.cuda.synchronize()
        return torch.cuda.mem_get_info()[0]

    first = [work() for _ in range(3)][-1]
    assert min(work() for _ in range(20)) >= first - (1 << 20)
    b = Batch(W, [5], 1, 64)
    b.cache.free()
    b.cache.free()  # no-op
    with pytest.raises(ValueError, match="freed"):
        b.everything()
