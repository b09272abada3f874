"""Device memory that the library keeps outside its pool."""
import os
import subprocess
import sys

import pytest

pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = r"""
import sys
import torch
sys.path.insert(0, sys.argv[1])
from decode_gemv_sign_gb300 import build, wcomp as W
build.build()
x = torch.randn(2, 4096, device="cuda").bfloat16()
weights = [W.q4_encode(torch.randn(N, 4096, device="cuda").bfloat16(), 64) for N in (64, 9744)]
W.q4_encode(torch.zeros(32768, 4096, dtype=torch.bfloat16, device="cuda"), 64).free()  # 72 MB that the pool keeps
y = [torch.empty(2, N, device="cuda") for N in (64, 9744)]
torch.cuda.synchronize()
before = torch.cuda.mem_get_info()[0]
for w, out in zip(weights, y):
    W.q4_gemv(w, x, out)
torch.cuda.synchronize()
print(before - torch.cuda.mem_get_info()[0])
"""


def test_products_keep_no_counters():
    """4-bit products alone keep an error word (and their code, a few MB), not the expert layer's 25 MB of counters."""
    r = subprocess.run([sys.executable, "-c", CHILD, ROOT], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-4000:]
    print(r.stdout)
    assert int(r.stdout.split()[-1]) < 12 << 20, r.stdout


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("shape", [(1, 1), (32, 256), (33, 257), (3, 40, 300)])
def test_the_size_of_a_held_weight(shape, group):
    """M * ceil(N / 32) * ceil(K / 256) blocks of 4096 bytes of codes and 16384 / group of scales, as the header says."""
    import torch

    from decode_gemv_sign_gb300 import build, wcomp

    build.build()
    c = wcomp.q4_encode(torch.zeros(*shape, dtype=torch.bfloat16, device="cuda"), group)
    M, N, K = (1, *shape)[-3:]
    assert c.info()["bytes"] == M * -(-N // 32) * -(-K // 256) * (4096 + 16384 // group)
