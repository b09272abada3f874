"""Which positions the rows of a call have: windows up to the largest number, and starts that do not fit the call."""
import numpy as np
import pytest

from test_gpu_kv4 import Batch, attend_matches, dev16, draw, ints, reported

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def W():
    from decode_gemv_sign_gb300 import build, wcomp

    build.build()
    wcomp.lib()
    return wcomp


@pytest.mark.parametrize("D,width", [(64, 7), (128, 7), (256, 7), (64, 1100), (128, 1100), (256, 1100)])
@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 64, 2 ** 31 - 200])
def test_windows_as_large_as_numbers_go(W, D, width, window):
    """They are no window, also for sequences that hold fewer tokens than the call has rows."""
    lengths, rows = [100, 300, 0, 65, 130], [103, 2, 5, 200, 130]
    b = Batch(W, lengths, 2, D, seed=1, width=width)
    q = draw((sum(rows), 4, D), np.random.default_rng(window % 1000), 1.5)
    attend_matches(W, b, q, rows, window=window)
    W.device_check()


BAD = [[0, 2, 1000], [5, 2, 0], [-7, 2, 4], [0, 1000, 4], [0, 2 ** 31 - 1, 2 ** 31 - 1], [-2 ** 31, -5, 3], [0, 3, 2], [0, 4, 5]]


@pytest.mark.parametrize("starts", BAD, ids=str)
@pytest.mark.parametrize("width", [2, 1100])
def test_starts_that_descend_or_leave_the_call_are_reported(W, starts, width):
    """By every call that takes them, whatever kernel it has; nothing is read or written outside."""
    b = Batch(W, [70, 30], 1, 64, width=width)
    q = torch.full((4 + 2 * 64, 2, 64), 1.0, dtype=torch.bfloat16, device="cuda")
    s = ints(starts)
    W.device_check()
    for mass in (None, torch.zeros(2, 1, b.width * 64, device="cuda")):
        out = torch.full_like(q, 7.0)
        W.kv4_attend(b.cache, q[64:68], b.table, b.len, s, out=out[64:68], mass=mass)
        reported(W)
        assert (out[:64] == 7.0).all() and (out[68:] == 7.0).all()
    k, v = (torch.full((4 + 128, 1, 64), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    W.kv4_read(b.cache, b.table, b.len, s, k=k[64:68], v=v[64:68])
    reported(W)
    for t in (k, v):
        assert (t[:64] == 7.0).all() and (t[68:] == 7.0).all()
    W.kv4_append(b.cache, k[64:68], v[64:68], b.table, b.len, s)
    reported(W)


def test_the_one_bad_pair_of_many_is_reported(W):
    """Anywhere in more starts than a block has threads, and whatever rows there are."""
    B = 3000
    b = Batch(W, [3] * B, 1, 64, width=1)
    q = dev16(draw((B, 1, 64), np.random.default_rng(1)))
    good = np.arange(B + 1)
    W.kv4_attend(b.cache, q, b.table, b.len, ints(good))
    W.kv4_append(b.cache, q, q, b.table, b.len, ints(good))
    W.device_check()
    for at in (0, 1, 700, 1500, B - 1, B):
        s = good.copy()
        s[at] += 1 if at == B else -1 if at == 0 else 2
        for call in (lambda: W.kv4_attend(b.cache, q, b.table, b.len, ints(s)),
                     lambda: W.kv4_read(b.cache, b.table, b.len, ints(s), rows=B),
                     lambda: W.kv4_append(b.cache, q, q, b.table, b.len, ints(s))):
            call()
            reported(W)


@pytest.mark.parametrize("starts", [[0, 0, 0], [0, 4, 4], [2, 2, 4], [1, 2, 3], [0, 0, 4], [0, 1, 2]], ids=str)
def test_starts_that_fit_are_not(W, starts):
    b = Batch(W, [70, 30], 1, 64)
    q = torch.full((4, 1, 64), 1.0, dtype=torch.bfloat16, device="cuda")
    W.kv4_attend(b.cache, q, b.table, b.len, ints(starts), mass=torch.zeros(2, 1, b.width * 64, device="cuda"))
    W.kv4_read(b.cache, b.table, b.len, ints(starts), rows=4)
    W.kv4_append(b.cache, q, q, b.table, b.len, ints(starts))
    W.device_check()
