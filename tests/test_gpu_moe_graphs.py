"""What captured expert layers take and give back: graphs made, run and destroyed through the driver's own calls."""
import ctypes
import time

import pytest

from test_gpu_moe import Layer, dev

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

P = ctypes.c_void_p


@pytest.fixture(scope="module")
def W():
    from decode_gemv_sign_gb300 import build, wcomp

    build.build()
    wcomp.lib()
    return wcomp


class Graph:
    """`calls` calls of call(stream) as an executable graph, and how many nodes they were."""

    def __init__(self, stream, call, calls=1):
        self.cuda, self.stream = ctypes.CDLL("libcuda.so.1"), P(stream.cuda_stream)
        graph, nodes, self.exec = P(), ctypes.c_size_t(), P()
        self.do("cuStreamBeginCapture_v2", self.stream, 2)  # relaxed
        for _ in range(calls):
            call(stream)
        self.do("cuStreamEndCapture", self.stream, ctypes.byref(graph))
        self.do("cuGraphGetNodes", graph, None, ctypes.byref(nodes))
        self.do("cuGraphInstantiateWithFlags", ctypes.byref(self.exec), graph, ctypes.c_ulonglong(0))
        self.do("cuGraphDestroy", graph)
        self.nodes = nodes.value

    def do(self, name, *args):
        assert getattr(self.cuda, name)(*args) == 0, name

    def launch(self):
        self.do("cuGraphLaunch", self.exec, self.stream)

    def destroy(self):
        self.do("cuGraphExecDestroy", self.exec)


@pytest.fixture(scope="module")
def layer(W):
    a = Layer(W, 1, 2, 8, 8, 32, seed=50)
    args = (dev(a.x), dev(a.router), *a.dev, 1)
    want = W.moe(*args)
    torch.cuda.synchronize()
    return args, want


def test_counters_come_back_with_their_graph(W, layer):
    """However many captured calls there have been, a new one is as many nodes as the first."""
    args, want = layer
    stream, y = torch.cuda.Stream(), torch.zeros_like(want)

    def call(s):
        W.moe(*args, y=y, stream=s)

    first = Graph(stream, call)
    for _ in range(6):
        g = Graph(stream, call, 1000)
        y.zero_()
        torch.cuda.synchronize()
        g.launch()
        g.destroy()  # under way
        stream.synchronize()
        assert torch.equal(y, want)
    for _ in range(100):  # the driver gives them back on a thread of its own
        again = Graph(stream, call)
        if again.nodes == first.nodes:
            break
        again.destroy()
        time.sleep(0.05)
    assert again.nodes == first.nodes
    for g in (first, again):
        y.zero_()
        torch.cuda.synchronize()
        g.launch()
        stream.synchronize()
        assert torch.equal(y, want)
        g.destroy()
    W.device_check()


def test_more_live_calls_than_sets(W, layer):
    """Calls beyond the kept sets clear counters of their own, a node more, and are right next to others."""
    args, want = layer
    streams = [torch.cuda.Stream() for _ in range(2)]
    ys = [torch.zeros_like(want) for _ in range(3)]
    many = Graph(streams[0], lambda s: W.moe(*args, y=ys[0], stream=s), 5400)
    over = Graph(streams[1], lambda s: W.moe(*args, y=ys[1], stream=s))
    few = over.nodes
    torch.cuda.synchronize()
    for _ in range(3):
        for y in ys:
            y.zero_()
        torch.cuda.synchronize()
        many.launch()
        for _ in range(200):
            over.launch()
            W.moe(*args, y=ys[2])
        torch.cuda.synchronize()
        assert all(torch.equal(y, want) for y in ys)
    many.destroy()
    over.destroy()
    for _ in range(100):
        g = Graph(streams[1], lambda s: W.moe(*args, y=ys[1], stream=s))
        g.destroy()
        if g.nodes < few:
            break
        time.sleep(0.05)
    assert g.nodes == few - 1  # without the clearing
    W.device_check()
