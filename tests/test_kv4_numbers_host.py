"""Numbers that the library's arguments do not hold are refused on the host."""
import pytest
import torch

from decode_gemv_sign_gb300 import wcomp
from test_kv4_host import cache, lib  # noqa: F401


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
