"""A process's first call on a stream that waits for nothing, while the default stream is busy.

The library sets its counters up on first use.  They have to be clear before
the first kernel reads them, on whatever stream that runs: torch's streams do
not wait for the default stream, behind whose work a clearing there would come
(a thread of the test keeps some of it queued).
Each operation makes the first call of a process of its own, after memory of
the size of the counters was filled with ones and given back to the driver.
"""
import os
import subprocess
import sys

import pytest

pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = r"""
import sys
import threading
import torch
sys.path.insert(0, sys.argv[1])
from decode_gemv_sign_gb300 import build, wcomp as W
build.build()
W.lib()
g = torch.Generator(device="cuda")
g.manual_seed(1)

def draw(*shape):
    return (torch.randn(*shape, device="cuda", generator=g) * 0.1).bfloat16()

if sys.argv[2] == "moe":
    args = [draw(4, 512), draw(16, 512), draw(16, 256, 512), draw(16, 256, 512), draw(16, 512, 256)]
    call = lambda: W.moe(*args, 4)
elif sys.argv[2] == "q4_gemv":  # rows cut over blocks and joined
    w, x = W.q4_encode(draw(9744, 14350), 64), draw(2, 14350)
    call = lambda: W.q4_gemv(w, x)
else:
    w, x = W.encode(draw(4096, 4096), "bytesplit"), draw(2, 4096)
    call = lambda: W.gemv(w, x)
junk = [torch.full((n,), -1, dtype=torch.int32, device="cuda") for n in (1 << 10, 1 << 12, 1 << 20, 1 << 23, 1 << 23)]
torch.cuda.synchronize()
del junk
torch.cuda.empty_cache()
side = torch.cuda.Stream()
# another thread keeps the default stream some 50 ms behind, also after calls that wait for the device
stop = threading.Event()
def feed():
    events = []
    for _ in range(1000):
        if stop.is_set():
            return
        torch.cuda._sleep(10_000_000)  # about 5 ms
        events.append(torch.cuda.Event())
        events[-1].record()
        if len(events) > 10:
            events[-10].synchronize()
feeder = threading.Thread(target=feed)
feeder.start()
with torch.cuda.stream(side):
    first = call()
    second = call()
side.synchronize()
stop.set()
feeder.join()
torch.cuda.synchronize()
W.device_check()
third = call()
assert torch.equal(first, second) and torch.equal(first, third)
assert torch.isfinite(first.float()).all() and first.float().abs().max() > 0
W.device_check()
print("ok")
"""


@pytest.mark.parametrize("op", ["moe", "q4_gemv", "gemv"])
def test_first_call_on_a_side_stream(op):
    r = subprocess.run([sys.executable, "-c", CHILD, ROOT, op], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.endswith("ok\n"), r.stdout[-2000:] + r.stderr[-4000:]
