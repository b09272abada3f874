"""The container GEMV next to itself: each launch has work counters that no other uses while it runs."""
import numpy as np
import pytest

from decode_gemv_sign_gb300 import synth
from oracle import wcomp_oracle as O

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


def test_a_graph_and_two_streams_next_to_many_calls(W):
    """A captured call runs as often as its graph does while more calls than there once were counters go by."""
    spec = synth.WeightSpec("s", 6144, 2048, "t4", 0.02, 0.001, "normal", 0.1, seed=3)
    w, x = synth.gen_weights_np(spec), synth.gen_x_np(2, 2048, 4)
    c, xd = W.encode(dev(w), "bytesplit"), dev(x)
    want = W.gemv(c, xd)
    y_ref = O.gemv(w, x)
    assert np.abs(want.cpu().numpy() - y_ref).max() <= 1e-4 * np.abs(y_ref).max()
    held, graph, side = torch.zeros_like(want), torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        W.gemv(c, xd, held)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for turn in range(4):
        out = [torch.zeros_like(want) for _ in range(600)]
        torch.cuda.synchronize()
        for i, y in enumerate(out):
            with torch.cuda.stream(streams[i % 2]):
                W.gemv(c, xd, y)
            with torch.cuda.stream(side):
                if i % 8 == 0:
                    held.zero_()
                graph.replay()
        torch.cuda.synchronize()
        W.device_check()
        assert torch.equal(held, want) and all(torch.equal(y, want) for y in out)
