"""Sizes whose product passes 64 bits are refused before any CUDA call (CPU only; the pointers are never
followed)."""
import ctypes

import pytest

from test_lm_refusals import P, cache, lib, refused  # noqa: F401


@pytest.mark.parametrize("B,T,heads", [(2 ** 30, 2 ** 30, 16), (2 ** 31 - 1, 2 ** 31 - 1, 65535), (2 ** 16, 2 ** 15, 1),
                                       (2 ** 15, 2 ** 14, 5)])
def test_cache_write(lib, B, T, heads):  # noqa: F811
    c = ctypes.byref(cache(kv_heads=heads))
    refused(lib, lib.fa_cache_write(c, 0, B, T, P, 64, 64, 64, P, 64, 64, 64, P, 2, P, None, None, None, 0, 0, 1.0, None))


@pytest.mark.parametrize("n,heads,dim", [(2 ** 58, 64, 64), (2 ** 63 - 1, 1, 1), (2 ** 32, 2 ** 31 - 1, 1024)])
def test_rope(lib, n, heads, dim):  # noqa: F811
    refused(lib, lib.fa_rope(0, n, heads, dim, 0, 0, 0, P, 128, 64, P, P, 1.0, P, 128, 64, None))
