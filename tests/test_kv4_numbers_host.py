"""Numbers that the library's arguments cannot hold, or its arithmetic cannot, are refused on the host."""
import ctypes

import pytest
import torch

from decode_gemv_sign_gb300 import wcomp
from test_kv4_host import cache, lib, logprob_args  # noqa: F401


@pytest.mark.parametrize("window", [-1, 2 ** 31, 2 ** 32, 2 ** 32 + 5])
def test_windows_beyond_32_bits_are_refused(window):
    c = cache("cpu")
    i32 = dict(dtype=torch.int32)
    q = torch.zeros(2, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="window"):
        wcomp.kv4_attend(c, q, torch.zeros(2, 4, **i32), torch.zeros(2, **i32), window=window)


@pytest.mark.parametrize("pages,heads,dim", [(4, 2 ** 32 + 8, 64), (4, 8, 2 ** 32 + 64), (4, 2 ** 31, 64),
                                             (4, -2 ** 32 + 8, 64), (2 ** 64 + 4, 8, 64)])
def test_cache_sizes_beyond_the_arguments_are_refused(lib, pages, heads, dim):  # noqa: F811
    with pytest.raises(ValueError, match="heads and dim"):
        wcomp.kv4_create(pages, heads, dim, stream=0)


def test_scales_whose_product_with_log2_e_overflows_are_refused(lib):  # noqa: F811
    for scale in (2.0 ** 127.5, 3e38, 3.4028234663852886e38):
        assert lib.wcomp_logprobs(ctypes.byref(logprob_args(scale=scale)), None) == wcomp.EINVAL, scale
    assert lib.wcomp_logprobs(ctypes.byref(logprob_args(scale=2.0 ** 127, T=0)), None) == wcomp.OK
    assert lib.wcomp_logprobs(ctypes.byref(logprob_args(scale=1e-45, T=0)), None) == wcomp.OK
