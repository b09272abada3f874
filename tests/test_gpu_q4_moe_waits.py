"""What happens when a bounded wait of the 4-bit and expert kernels runs out.

Under the debug build, whose hooks leave a copy unissued or let a thread block
come late to a grid barrier (nothing faults, every wait has its limit): the call
finishes, wcomp_device_check reports WCOMP_ETIMEOUT, and no other call is
touched: not the next one on the same counters, whether or not the error was
taken in between, and not one that runs while it is taken.
"""
import os
import subprocess
import sys

import pytest

pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

COMMON = r"""
import sys, time
import torch
sys.path.insert(0, sys.argv[1])
from decode_gemv_sign_gb300 import wcomp as W
W.LIB_PATH = sys.argv[2]
L = W.lib()
g = torch.Generator(device="cuda")
g.manual_seed(1)

def draw(*shape):
    return (torch.randn(*shape, device="cuda", generator=g) * 0.1).bfloat16()

def layer(T, E, H, F, group):
    ws = [draw(E, F, H), draw(E, F, H), draw(E, H, F)]
    return [draw(T, H), draw(E, H), *([W.q4_encode(w, group) for w in ws] if group else ws)]

def run_out(hook, call):
    # the call under a hook, which makes one of its waits run out
    assert L.wcomp_debug_skip_first_copy(hook) == W.OK
    t0 = time.time()
    call()
    torch.cuda.synchronize()
    dt = time.time() - t0
    assert 0.5 < dt < 30, dt
    assert L.wcomp_debug_skip_first_copy(0) == W.OK

assert L.wcomp_device_check(None) == W.OK
"""

COPIES = COMMON + r"""
calls = []
# records of x in the blocks; whole units; clusters; rows cut and joined; the same for 16 rows of x
for N, K, B, group in ((512, 2048, 1, 128), (4096, 4096, 8, 64), (256, 20000, 3, 32), (9744, 14350, 2, 64), (256, 20000, 16, 32),
                       (9744, 14350, 16, 128)):
    w, x = W.q4_encode(draw(N, K), group), draw(B, K)
    calls.append((f"gemv {N} {K} {B}", lambda w=w, x=x: W.q4_gemv(w, x)))
for T, E, H, F, group in ((1, 4, 1024, 512, 0), (16, 4, 1024, 512, 0), (1, 4, 1024, 512, 64), (16, 4, 1000, 333, 32)):
    a = layer(T, E, H, F, group)
    calls.append((f"moe {T} {E} {H} {F} {group}", lambda a=a: W.moe(*a, 2)))
for name, call in calls:
    want = call()
    run_out(1, call)
    assert L.wcomp_device_check(None) == W.ETIMEOUT, name
    assert L.wcomp_device_check(None) == W.OK, name
    assert torch.equal(call(), want), name
    assert L.wcomp_device_check(None) == W.OK, name
    print("recovered", name)
"""

LATE = COMMON + r"""
# gate and up rows of a few units, cut over many blocks and joined; the same layers through odd widths
for T, E, H, F, group in ((1, 2, 8192, 40, 0), (1, 2, 8191, 41, 0), (1, 2, 8192, 40, 32), (12, 2, 8192, 40, 128)):
    a = layer(T, E, H, F, group)
    want = W.moe(*a, 1)
    y = torch.empty_like(want)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        W.moe(*a, 1, y=y)
    for name, call in (("graph", lambda: graph.replay()), ("call", lambda: W.moe(*a, 1, y=y))):
        run_out(2, call)
        for _ in range(1100):  # every set of counters in turn; the error is not taken before
            y.zero_()
            call()
            assert torch.equal(y, want), (T, H, F, group, name)
        assert L.wcomp_device_check(None) == W.ETIMEOUT
        assert L.wcomp_device_check(None) == W.OK
        print("recovered", T, H, F, group, name)
"""

CHECK_NEXT_TO_CALLS = COMMON + r"""
w, x = W.q4_encode(draw(512, 2048), 128), draw(1, 2048)
layers = [layer(T, 16, 1024, 512, group) for T, group in ((2, 0), (4, 64))]
want = [W.moe(*a, 4) for a in layers]
y = torch.empty_like(want[0])
graph = torch.cuda.CUDAGraph()
torch.cuda.synchronize()
with torch.cuda.graph(graph):
    W.moe(*layers[0], 4, y=y)
for turn in range(3):
    run_out(1, lambda: W.q4_gemv(w, x))
    streams = [torch.cuda.Stream() for _ in layers]
    got = [[] for _ in layers]
    y.zero_()
    under_way = torch.cuda.Event()
    for s in streams:
        with torch.cuda.stream(s):
            torch.cuda._sleep(100_000_000)  # 50 ms, in which the calls are queued
    for i in (1, 0):
        with torch.cuda.stream(streams[i]):
            for _ in range(100):
                got[i].append(W.moe(*layers[i], 4))
                if i == 0 and len(got[0]) == 5:
                    under_way.record()
            if i == 0:
                for _ in range(100):
                    graph.replay()
    under_way.synchronize()
    assert not streams[0].query()  # they are still at it
    assert L.wcomp_device_check(None) == W.ETIMEOUT
    torch.cuda.synchronize()
    assert L.wcomp_device_check(None) == W.OK
    for i in range(len(layers)):
        assert all(torch.equal(t, want[i]) for t in got[i])
    assert torch.equal(y, want[0])
    print("untouched", turn)
"""


def run(child, word, times):
    from decode_gemv_sign_gb300 import build

    lib = build.build(debug=True)
    r = subprocess.run([sys.executable, "-c", child, ROOT, lib], capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-4000:]
    assert r.stdout.count(word) == times


def test_copies_that_never_arrive():
    run(COPIES, "recovered", 10)


def test_a_block_that_comes_late_to_a_barrier():
    run(LATE, "recovered", 8)


def test_the_check_next_to_running_calls():
    run(CHECK_NEXT_TO_CALLS, "untouched", 3)
