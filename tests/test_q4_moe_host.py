"""The 4-bit and expert entry points refuse bad arguments on the host, before any CUDA call, and the
definitions that the GPU tests compare against are pinned to values worked out by hand."""
import ctypes

import numpy as np
import pytest
import torch

from decode_gemv_sign_gb300 import wcomp
from oracle import q4_moe_oracle as Q

P = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    from decode_gemv_sign_gb300 import build

    build.build()
    return wcomp.lib()


def test_q4_argument_errors_without_gpu(lib):
    h = P(1)
    ok = P(256)
    assert lib.wcomp_q4_encode(None, 1, 4, 4, 32, None, ctypes.byref(h)) == wcomp.EINVAL
    assert not h.value  # the output is cleared
    assert lib.wcomp_q4_encode(ok, 1, 4, 4, 32, None, None) == wcomp.EINVAL
    for M, N, K, g in ((0, 4, 4, 32), (1, 0, 4, 32), (1, 4, -1, 32), (1, 4, 4, 48), (1, 4, 4, 0)):
        assert lib.wcomp_q4_encode(ok, M, N, K, g, None, ctypes.byref(h)) == wcomp.EINVAL
        assert lib.wcomp_q4_pack(ok, ok, M, N, K, g, None, ctypes.byref(h)) == wcomp.EINVAL
    for M, N, K in ((1, 1 << 31, 4), (1, 4, 1 << 31), (1 << 31, 4, 4), (1 << 20, 1 << 20, 4),
                    (1 << 15, 1 << 16, 1 << 30)):
        assert lib.wcomp_q4_encode(ok, M, N, K, 32, None, ctypes.byref(h)) == wcomp.EUNSUPPORTED
    assert lib.wcomp_q4_pack(None, ok, 1, 4, 4, 32, None, ctypes.byref(h)) == wcomp.EINVAL
    assert lib.wcomp_q4_pack(ok, None, 1, 4, 4, 32, None, ctypes.byref(h)) == wcomp.EINVAL
    assert lib.wcomp_q4_decode(None, ok, None) == wcomp.EINVAL
    assert lib.wcomp_q4_unpack(None, ok, ok, None) == wcomp.EINVAL
    assert lib.wcomp_q4_gemv(None, ok, 1, ok, None) == wcomp.EINVAL
    assert lib.wcomp_q4_info(None, None) == wcomp.EINVAL
    lib.wcomp_q4_free(None, None)  # no-op


def args(**kw):
    a = wcomp.MoeArgs()
    for n in ("d_x", "d_router", "d_gate", "d_up", "d_down", "d_y"):
        setattr(a, n, 256)
    a.H, a.F, a.T, a.E, a.top_k, a.scoring, a.factor = 64, 32, 1, 4, 2, 0, 1.0
    for n, v in kw.items():
        setattr(a, n, v)
    return a


def test_moe_argument_errors_without_gpu(lib):
    assert lib.wcomp_moe(None, None) == wcomp.EINVAL
    for bad in (dict(d_x=None), dict(d_router=None), dict(d_y=None), dict(T=0), dict(T=17), dict(E=0), dict(top_k=0),
                dict(top_k=5), dict(H=0), dict(F=0), dict(scoring=2), dict(scoring=-1)):
        assert lib.wcomp_moe(ctypes.byref(args(**bad)), None) == wcomp.EINVAL, bad
    for bad in (dict(E=1025), dict(E=100, top_k=17), dict(H=(1 << 24) + 1), dict(F=(1 << 24) + 1)):
        assert lib.wcomp_moe(ctypes.byref(args(**bad)), None) == wcomp.EUNSUPPORTED, bad


def test_the_binding_mirrors_the_header_structs(lib):
    # twelve pointers, two int64, five int32 and a float
    assert ctypes.sizeof(wcomp.MoeArgs) == 12 * 8 + 2 * 8 + 6 * 4
    assert ctypes.sizeof(wcomp.Q4Info) == 3 * 8 + 2 * 4 + 8


def test_host_tensors_are_refused():
    w = torch.zeros(4, 32, dtype=torch.bfloat16)
    with pytest.raises(TypeError, match="CUDA tensor"):
        wcomp.q4_encode(w)
    with pytest.raises(TypeError, match="CUDA"):
        wcomp.q4_pack(torch.zeros(4, 16, dtype=torch.uint8), w, 32, 32)
    with pytest.raises(TypeError, match="CUDA tensor"):
        wcomp.moe(w, w, w, w, w, 1)


def test_bf16_rounding_of_the_oracle():
    v = np.array([0.0, 1.0, -2.0, 1 + 2.0 ** -8, 1 + 3 * 2.0 ** -8, 1 + 2.0 ** -8 + 2.0 ** -40, 3.4e38, 1e39, np.inf,
                  2.0 ** -133, 2.0 ** -134, 1.5 * 2.0 ** -133])
    want = [0x0000, 0x3F80, 0xC000, 0x3F80, 0x3F82, 0x3F81, 0x7F80, 0x7F80, 0x7F80, 0x0001, 0x0000, 0x0002]
    assert [int(b) for b in Q.bf16(v)] == want
    r = np.random.default_rng(0).standard_normal(10000).astype(np.float32)
    assert np.array_equal(Q.bf16(r), torch.from_numpy(r).to(torch.bfloat16).view(torch.int16).numpy().view(np.uint16))


def test_q4_definition_by_hand():
    # the largest magnitude is 7: scale 1, values round half to even
    w = Q.bf16(np.array([[7.0, 0.5, 1.5, -2.5, 6.5, -6.49, 0.0, -7.0]]))
    codes, scales = Q.q4_encode(w, 32)
    assert scales.tolist() == [[0x3F80]]
    assert codes.tolist() == [[15, 8, 10, 6, 14, 2, 8, 1]]  # -6.49 is -6.5 in BF16: to the even -6
    assert Q.q4_values(codes, scales, 32).tolist() == [[7, 0, 2, -2, 6, -6, 0, -7]]
    assert Q.pack_codes(codes).tolist() == [[0x8F, 0x6A, 0x2E, 0x18]]
    assert Q.pack_codes(codes[:, :3]).tolist() == [[0x8F, 0x8A]]


def test_moe_definition_by_hand():
    one = Q.bf16(np.ones((1, 1)))
    g = np.full((2, 1, 1), 2.0)
    u = np.array([[[3.0]], [[5.0]]])
    d = np.ones((2, 1, 1))
    y, tol = Q.moe(one, g, u, d, np.array([[1, 0]]), np.array([[0.25, 0.75]]))
    s = 2.0 / (1.0 + np.exp(-2.0))
    assert np.isclose(y[0, 0], s * (0.25 * 5 + 0.75 * 3)) and 0 < tol[0, 0] < 0.01 * y[0, 0]
