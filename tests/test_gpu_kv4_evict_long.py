"""Eviction from long sequences, against its definition: weights beyond a block's registers, beyond its shared memory,
and over the blocks of a cluster; and from tables with pages that do not exist."""
import numpy as np
import pytest

from oracle import kv4_oracle as K
from test_gpu_kv4 import Batch, bits, dev16, draw, ints, reported, same_values

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def W():
    from decode_gemv_sign_gb300 import build, wcomp

    build.build()
    wcomp.lib()
    return wcomp


def masses(kind, shape, seed):
    rng = np.random.default_rng(seed)
    if kind == "random":
        m = rng.random(shape) ** 4
    elif kind == "ties":  # long runs of equal weights, few of which are taken, over every border
        m = np.repeat(rng.integers(0, 4, (*shape[:-1], -(-shape[-1] // 5000))), 5000, -1)[..., :shape[-1]] / 4.0
    elif kind == "equal":
        m = np.full(shape, 0.25)
    else:  # mostly NaN, the others anywhere, infinities and zeros of both signs among them
        m = np.full(shape, np.nan)
        pick = rng.random(shape) < 0.001
        m[pick] = rng.choice([0.0, -0.0, 1.0, np.inf, -np.inf, -1e-45], pick.sum())
    return m.astype(np.float32)


def evicts(W, lengths, width, H, kind, keep, recent, seed=0):
    """Sequences that share the pages of one run of tokens: choice, weights and what is moved."""
    D, B = 64, len(lengths)
    base = Batch(W, [4000], H, D, seed=seed)
    pages = base.table_np[0, :62]
    wide = -(-keep // 64)
    cache = W.kv4_create(base.pages + B * wide, H, D)
    W.kv4_append(cache, dev16(base.k), dev16(base.v), base.table, base.len, ints([0, 4000]))
    table = ints(np.tile(np.resize(pages, width), (B, 1)))
    out = ints(base.pages + np.random.default_rng(seed).permutation(B * wide).reshape(B, wide))
    m = masses(kind, (B, H, width * 64), seed)
    kept = torch.empty(B, H, keep, dtype=torch.int32, device="cuda")
    n, mass = W.kv4_evict(cache, table, ints(lengths), torch.from_numpy(m).cuda(), keep, recent, out, kept=kept)
    assert n.tolist() == [min(x, keep) for x in lengths]
    k, v = W.kv4_read(cache, base.table, base.len, ints([0, 4000]), rows=4000)
    kept, mass = kept.cpu().numpy(), mass.cpu().numpy()
    for i, x in enumerate(lengths):
        held = min(x, keep)
        got = W.kv4_read(cache, out[i:i + 1].contiguous(), n[i:i + 1], ints([0, held]), rows=held)
        for h in range(H):
            want = K.evict(m[i, h], x, keep, recent)
            assert np.array_equal(kept[i, h, :held], want), (i, h)
            assert (kept[i, h, held:] == -1).all() and (mass[i, h, held:] == 0).all()
            assert np.array_equal(mass[i, h, :held], m[i, h, want], equal_nan=True)
            at = torch.from_numpy(want % (62 * 64)).cuda()
            assert torch.equal(got[0][:, h], k[at, h]) and torch.equal(got[1][:, h], v[at, h])
    W.device_check()


# A block holds 8192 weights in registers and 11264 in shared memory; above 19456 places up to 8 blocks share a sequence
# and head while there are few of them.
@pytest.mark.parametrize("kind", ["random", "ties", "equal", "nan"])
@pytest.mark.parametrize("lengths", [[8191, 8193], [9000], [19456, 500, 0, 16000], [19457], [20000, 9999, 1, 64],
                                     [50000, 39000], [160001, 77, 12345], [400000, 123457]], ids=str)
def test_long_sequences(W, lengths, kind):
    width = -(-max(lengths) // 64)
    evicts(W, lengths, width, 2, kind, 777, 100, seed=len(lengths))
    evicts(W, lengths, width, 1, kind, max(lengths) - 3, 0, seed=1)
    evicts(W, lengths, width, 1, kind, max(lengths) // 2, max(lengths) // 2 - 1, seed=2)


@pytest.mark.parametrize("kind", ["random", "ties"])
def test_long_sequences_of_a_large_batch(W, kind):
    """So many that one block has each: weights beyond its shared memory are read again."""
    rng = np.random.default_rng(3)
    lengths = [int(n) for n in rng.integers(0, 30001, 160)]
    lengths[7], lengths[100] = 30000, 19457
    evicts(W, lengths, 469, 2, kind, 300, 20)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_tokens_of_pages_that_do_not_exist_become_zeros(W, D):
    """What is kept of them is rows of zeros, not what the output pages held before."""
    b = Batch(W, [200, 130], 2, D, width=4, spare=6)
    free = [p for p in range(b.pages) if p not in set(b.table_np.flatten())]
    out = ints(np.array(free[:4]).reshape(2, 2))
    junk = dev16(draw((256, 2, D), np.random.default_rng(1)))
    rng = np.random.default_rng(2)
    m = rng.random((2, 2, 256)).astype(np.float32)
    for page in (-1, b.pages, 2 ** 31 - 1, -2 ** 31):
        W.kv4_append(b.cache, junk, junk, out, ints([128, 128]), ints([0, 128, 256]))
        W.device_check()
        table = b.table.clone()
        table[0, 1] = page
        kept = torch.empty(2, 2, 100, dtype=torch.int32, device="cuda")
        n, mass = W.kv4_evict(b.cache, table, b.len, torch.from_numpy(m).cuda(), 100, 10, out, kept=kept)
        reported(W)
        k, v = (bits(t).reshape(2, 100, 2, D) for t in W.kv4_read(b.cache, out, n, ints([0, 100, 200]), rows=200))
        for i, x in enumerate(b.lengths):
            for h in range(2):
                want = K.evict(m[i, h], x, 100, 10)
                assert np.array_equal(kept[i, h].cpu().numpy(), want)
                assert np.array_equal(mass[i, h, :100].cpu().numpy(), m[i, h, want])
                there = ((want // 64 != 1) | (i == 1))[:, None]
                same_values(k[i, :, h], np.where(there, b.ks[i][want, h], 0.0))
                same_values(v[i, :, h], np.where(there, b.vs[i][want, h], 0.0))
        W.device_check()
