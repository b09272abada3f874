"""A call that fails leaves nothing behind for the next one."""
import ctypes

import numpy as np
import pytest

from decode_gemv_sign_gb300 import synth
from oracle import q4_moe_oracle as Q

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def W():
    from decode_gemv_sign_gb300 import build, wcomp

    build.build()
    wcomp.lib()
    return wcomp


def out_of_memory(W, x):
    """Weights of 2^58 values: their memory is refused before anything is read."""
    h = ctypes.c_void_p(1)
    st = W.lib().wcomp_q4_encode(x.data_ptr(), 1, 1 << 30, 1 << 28, 128, None, ctypes.byref(h))
    assert st == W.ENOMEM and not h.value
    st = W.lib().wcomp_q4_pack(x.data_ptr(), x.data_ptr(), 1, 1 << 30, 1 << 28, 128, None, ctypes.byref(h))
    assert st == W.ENOMEM and not h.value


def test_calls_after_a_weight_that_found_no_memory(W):
    w = synth.gen_weights_np(synth.WeightSpec("e", 64, 512, "t4", 0.02, 0.001, "normal", 0.1, seed=5))
    wd = torch.from_numpy(w.view(np.int16)).cuda()
    xd = torch.from_numpy(synth.gen_x_np(2, 512, 3).view(np.int16)).cuda()
    c, lossless = W.q4_encode(wd, 64), W.encode(wd, "bytesplit")
    y, z = W.q4_gemv(c, xd), W.gemv(lossless, xd)
    layer = [xd, wd[:4], wd.view(4, 16, 512), wd.view(4, 16, 512), wd.view(4, 512, 16)]
    m = W.moe(*layer, 2)
    codes, scales = Q.q4_encode(w, 64)
    calls = [
        lambda: np.array_equal(W.q4_unpack(W.q4_encode(wd, 64))[0].cpu().numpy(), Q.pack_codes(codes)),
        lambda: np.array_equal(W.q4_unpack(c)[0].cpu().numpy(), Q.pack_codes(codes)),
        lambda: W.q4_decode(c).shape == wd.shape,
        lambda: torch.equal(W.q4_gemv(c, xd), y),
        lambda: torch.equal(W.moe(*layer, 2), m),
        lambda: torch.equal(W.gemv(lossless, xd), z),
        lambda: torch.equal(W.decode(lossless), wd),
        lambda: torch.equal(W.decode(W.encode(wd, "k15")), wd),
    ]
    for call in calls:
        out_of_memory(W, xd)
        assert call()
    W.device_check()
