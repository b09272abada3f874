"""The calls on a 4-bit key/value cache and logprobs refuse bad arguments on the host, before any CUDA call, and the
definitions that the GPU tests compare against are pinned to values worked out by hand."""
import ctypes

import numpy as np
import pytest
import torch

from decode_gemv_sign_gb300 import wcomp
from oracle import kv4_oracle as K
from oracle.q4_moe_oracle import bf16

P = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    from decode_gemv_sign_gb300 import build

    build.build()
    return wcomp.lib()


def seqs(**kw):
    s = wcomp.Kv4Seqs(256, 256, None, 2, 4)
    for n, v in kw.items():
        setattr(s, n, v)
    return s


def test_create_refuses_bad_sizes(lib):
    h = P(1)
    for pages, heads, dim in ((0, 1, 64), (-1, 1, 64), (1, 0, 64), (1, 1, 0), (1, 1, -64)):
        assert lib.wcomp_kv4_create(pages, heads, dim, None, ctypes.byref(h)) == wcomp.EINVAL
        assert not h.value  # the output is cleared
    for pages, heads, dim in ((1, 1, 32), (1, 1, 96), (1, 1, 512), (1 << 31, 1, 64), (1 << 20, 1 << 11, 64),
                              (1, 1 << 16, 64)):
        assert lib.wcomp_kv4_create(pages, heads, dim, None, ctypes.byref(h)) == wcomp.EUNSUPPORTED
    assert lib.wcomp_kv4_create(1, 1, 64, None, None) == wcomp.EINVAL
    assert lib.wcomp_kv4_info(None, None) == wcomp.EINVAL
    lib.wcomp_kv4_free(None, None)  # no-op


def test_null_caches_are_refused(lib):
    s, ok = seqs(), P(256)
    assert lib.wcomp_kv4_append(None, ctypes.byref(s), ok, 64, 64, ok, 64, 64, 2, None) == wcomp.EINVAL
    assert lib.wcomp_kv4_read(None, ctypes.byref(s), ok, ok, 2, None) == wcomp.EINVAL
    assert lib.wcomp_kv4_attend(None, None, None) == wcomp.EINVAL
    assert lib.wcomp_kv4_attend(None, ctypes.byref(wcomp.Kv4AttendArgs(s)), None) == wcomp.EINVAL
    assert lib.wcomp_kv4_evict(None, None, None) == wcomp.EINVAL
    assert lib.wcomp_kv4_evict(None, ctypes.byref(wcomp.Kv4EvictArgs()), None) == wcomp.EINVAL


def logprob_args(**kw):
    a = wcomp.LogprobsArgs(256, 256, 256, 256, None, 256, 256, 3, 100, 100, 0, 5, 1.0)
    for n, v in kw.items():
        setattr(a, n, v)
    return a


def test_logprobs_argument_errors_without_gpu(lib):
    assert lib.wcomp_logprobs(None, None) == wcomp.EINVAL
    for bad in (dict(d_logits=None), dict(d_logprob=None), dict(T=-1), dict(V=0), dict(row=99), dict(dtype=2),
                dict(dtype=-1), dict(top_k=-1), dict(top_k=101), dict(d_top_ids=None), dict(d_top_logprobs=None),
                dict(d_logits=258), dict(d_ids=260), dict(d_logprob=257), dict(d_entropy=258), dict(d_top_ids=258),
                dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf"))):
        assert lib.wcomp_logprobs(ctypes.byref(logprob_args(**bad)), None) == wcomp.EINVAL, bad
    for bad in (dict(top_k=65), dict(V=1 << 31, row=1 << 31)):
        assert lib.wcomp_logprobs(ctypes.byref(logprob_args(**bad)), None) == wcomp.EUNSUPPORTED, bad
    assert lib.wcomp_logprobs(ctypes.byref(logprob_args(T=0, d_logits=None)), None) == wcomp.OK


def test_the_binding_mirrors_the_header_structs(lib):
    assert ctypes.sizeof(wcomp.Kv4Info) == 8 + 2 * 4 + 8
    assert ctypes.sizeof(wcomp.Kv4Seqs) == 3 * 8 + 2 * 4
    # the sequences, q and its strides, three outputs, T, three 32-bit values and padding
    assert ctypes.sizeof(wcomp.Kv4AttendArgs) == 32 + 3 * 8 + 3 * 8 + 8 + 3 * 4 + 4
    assert ctypes.sizeof(wcomp.Kv4EvictArgs) == 7 * 8 + 5 * 4 + 4
    assert ctypes.sizeof(wcomp.LogprobsArgs) == 7 * 8 + 3 * 8 + 3 * 4 + 4


def cache(device="cuda:0"):
    c = wcomp.KV4(0, 8, 2, 64, torch.device(device))
    return c


def test_host_tensors_and_wrong_shapes_are_refused():
    """Nothing here reaches a device: every check comes before the library is called."""
    c = cache("cpu")  # stands for a cache of another device than the tensors' own
    i32 = dict(dtype=torch.int32)
    table, lengths, k = torch.zeros(2, 4, **i32), torch.zeros(2, **i32), torch.zeros(2, 2, 64, dtype=torch.bfloat16)
    on_gpu = cache()
    with pytest.raises(ValueError, match="table"):
        wcomp.kv4_append(on_gpu, k, k, table, lengths)
    with pytest.raises(ValueError, match="table"):
        wcomp.kv4_append(c, k, k, table.long(), lengths)
    with pytest.raises(ValueError, match="table"):
        wcomp.kv4_append(c, k, k, table[0], lengths)
    with pytest.raises(ValueError, match="table"):
        wcomp.kv4_append(c, k, k, torch.zeros(2, 8, **i32)[:, ::2], lengths)
    with pytest.raises(ValueError, match="lengths"):
        wcomp.kv4_append(c, k, k, table, lengths[:1])
    with pytest.raises(ValueError, match="starts"):
        wcomp.kv4_append(c, k, k, table, lengths, lengths)
    with pytest.raises(TypeError, match="BF16"):
        wcomp.kv4_append(c, k.float(), k, table, lengths)
    with pytest.raises(ValueError, match="v must be"):
        wcomp.kv4_append(c, k, k[:, :1], table, lengths)
    with pytest.raises(ValueError, match="contiguous columns"):
        wcomp.kv4_append(c, torch.zeros(2, 2, 128, dtype=torch.bfloat16)[..., ::2], k, table, lengths)
    with pytest.raises(ValueError, match="same rows"):
        wcomp.kv4_append(c, k, k[:1], table, lengths)
    with pytest.raises(ValueError, match="same rows"):
        wcomp.kv4_append(c, k[:1], k[:1], table, lengths)
    with pytest.raises(ValueError, match="rows must be given"):
        wcomp.kv4_read(c, table, lengths, torch.zeros(3, **i32))
    with pytest.raises(ValueError, match="one row a sequence"):
        wcomp.kv4_read(c, table, lengths, rows=3)
    with pytest.raises(ValueError, match="multiple of the cache's heads"):
        wcomp.kv4_attend(c, torch.zeros(2, 3, 64, dtype=torch.bfloat16), table, lengths)
    with pytest.raises(ValueError, match="one row a sequence"):
        wcomp.kv4_attend(c, k[:1], table, lengths)
    with pytest.raises(ValueError, match="q must be"):
        wcomp.kv4_attend(c, torch.zeros(2, 2, 128, dtype=torch.bfloat16), table, lengths)
    mass = torch.zeros(2, 2, 256)
    for keep, recent, out in ((0, 0, table), (4, 5, table), (4, -1, table), (257, 0, table)):
        with pytest.raises(ValueError, match="keep must be"):
            wcomp.kv4_evict(c, table, lengths, mass, keep, recent, out)
    with pytest.raises(ValueError, match="mass"):
        wcomp.kv4_evict(c, table, lengths, mass[..., :255], 4, 0, table.clone())
    with pytest.raises(ValueError, match="freed"):
        wcomp.kv4_append(c, k, k, table, lengths)
    with pytest.raises(TypeError, match="CUDA tensor"):
        wcomp.logprobs(torch.zeros(2, 4))


def test_attention_definition_by_hand():
    # scores log 1, log 3 for the second row; the first sees one token
    k = np.zeros((2, 1, 64))
    k[1, 0, 0] = 1.0
    v = np.zeros((2, 1, 64))
    v[:, 0, 5] = (2.0, 6.0)
    q = np.zeros((2, 1, 64))
    q[:, 0, 0] = 2 * np.log(3.0)
    out, lse, mass, out_tol, _, _ = K.attend(q, k, v, 0.5)
    assert np.allclose(out[:, 0, 5], [2.0, 0.25 * 2 + 0.75 * 6]) and np.allclose(lse[:, 0], [0.0, np.log(4.0)])
    assert np.allclose(mass, [[1.25, 0.75]]) and (out_tol[:, 0, 5] < 0.03).all()
    out, lse, mass, _, _, _ = K.attend(q, k, v, 0.5, window=1)
    assert np.allclose(out[:, 0, 5], [2.0, 6.0]) and np.allclose(mass, [[1.0, 1.0]])
    out, lse, mass, _, _, _ = K.attend(np.zeros((4, 1, 64)), k, v, 0.5)  # more rows than tokens
    assert (out[:2] == 0).all() and np.isneginf(lse[:2]).all() and np.allclose(mass, [[1.5, 0.5]])


def test_held_values_by_hand():
    w = np.zeros((1, 64))
    w[0, :4] = (7.0, 0.5, 1.5, -2.5)
    w[0, 32] = 14.0
    assert K.held(bf16(w))[0, [0, 1, 2, 3, 32, 33]].tolist() == [7, 0, 2, -2, 14, 0]


def test_eviction_definition_by_hand():
    m = np.array([1.0, 5.0, 5.0, np.nan, -np.inf, 0.0, 9.0])
    assert K.evict(m, 7, 7, 0).tolist() == [0, 1, 2, 3, 4, 5, 6]
    assert K.evict(m, 7, 3, 1).tolist() == [1, 2, 6]
    assert K.evict(m, 7, 2, 0).tolist() == [1, 6]
    assert K.evict(m, 7, 6, 1).tolist() == [0, 1, 2, 4, 5, 6]
    assert K.evict(m, 6, 1, 1).tolist() == [5]


def test_logprob_definition_by_hand():
    z = np.log(np.array([[1.0, 2.0, 1.0, 4.0], [0.0, 1.0, 1.0, 0.0]]))
    lp, ent, lse, top, ids, _ = K.logprobs(z, [1, -5], 3)
    assert np.allclose(lp, [np.log(0.25), 0.0]) and np.allclose(lse, np.log([8.0, 2.0]))
    assert np.allclose(ent, [0.25 * np.log(8) + 0.25 * np.log(4) + 0.5 * np.log(2), np.log(2.0)])
    assert ids.tolist() == [[3, 1, 0], [1, 2, 0]] and np.allclose(top[1, :2], np.log(0.5)) and np.isneginf(top[1, 2])
    lp, ent, _, top, ids, _ = K.logprobs(np.array([[-np.inf, -np.inf], [np.nan, 1.0]]), [0, 1], 1)
    assert np.isnan(lp).all() and np.isnan(ent).all() and ids.tolist() == [[0], [1]]
