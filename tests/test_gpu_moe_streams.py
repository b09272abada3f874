"""The expert layer on many streams at once: each launch has counters that no other uses while it runs."""
import ctypes

import pytest

from test_gpu_moe import Layer, dev

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def W():
    from decode_gemv_sign_gb300 import build, wcomp

    build.build()
    wcomp.lib()
    return wcomp


@pytest.fixture(scope="module")
def layers(W):
    out = []
    for T, form in ((2, "bf16"), (5, 64)):
        a = Layer(W, T, 16, 512, 256, form, seed=40 + T)
        args = (dev(a.x), dev(a.router), *a.dev, 4)
        out.append((args, W.moe(*args)))
    torch.cuda.synchronize()
    return out


@pytest.mark.parametrize("ahead", [1023, 1024, 2048])
def test_a_stream_behind_one_that_is_many_calls_ahead(W, layers, ahead):
    """A call that waits on its stream while another stream makes `ahead` calls and more: both run at the end."""
    (args, want), (other, also) = layers
    slow, fast = torch.cuda.Stream(), torch.cuda.Stream()
    with torch.cuda.stream(slow):
        torch.cuda._sleep(60_000_000)  # 30 ms: longer than the other stream's calls take to be queued
        got = [W.moe(*args) for _ in range(20)]
    with torch.cuda.stream(fast):
        y = [W.moe(*other) for _ in range(ahead)][-10:]
        if ahead == 2048:
            fast.wait_stream(slow)
        y += [W.moe(*other) for _ in range(40)]
    torch.cuda.synchronize()
    W.device_check()
    assert all(torch.equal(t, want) for t in got) and all(torch.equal(t, also) for t in y)


def test_more_streams_than_sets_of_counters(W, layers):
    cudart = torch.cuda.cudart()
    handles = []
    try:
        for i in range(1100):
            h = ctypes.c_void_p()
            assert int(cudart.cudaStreamCreate(ctypes.addressof(h))) == 0
            handles.append(h.value)
        for turn in range(2):
            got = []
            for i, h in enumerate(handles):
                args, want = layers[i % 2]
                y = torch.empty_like(want)
                W.moe(*args, y=y, stream=h)
                got.append((y, want))
            torch.cuda.synchronize()
            W.device_check()
            assert all(torch.equal(a, b) for a, b in got)
    finally:
        torch.cuda.synchronize()
        for h in handles:
            cudart.cudaStreamDestroy(h)
    # the streams that came first keep their sets, new ones do without
    for s in (None, torch.cuda.Stream()):
        args, want = layers[1]
        y = W.moe(*args, stream=s)
        torch.cuda.synchronize()
        assert torch.equal(y, want)
