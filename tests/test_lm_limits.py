"""The limits of the attention and of the cache reader that keep their indices in range, refused before
any CUDA call (CPU only; the pointers are never followed)."""
import ctypes
import math

import pytest

from test_lm_refusals import P, cache, lib, refused  # noqa: F401


def attend(lib, c, B=1, T=1, heads=2, max_pages=2, scale=1.0):  # noqa: F811
    return lib.fa_tree_attention(ctypes.byref(c), 1, B, T, heads, P, 64, 64, 64, P, max_pages, P, None, None, scale, P, None, P,
                                 1 << 40, None)


@pytest.mark.parametrize("scale", [0.0, -1.0, math.inf, -math.inf, math.nan])
def test_scale(lib, scale):  # noqa: F811
    refused(lib, attend(lib, cache(), scale=scale))


def test_slots_rows_and_tiles(lib):  # noqa: F811
    refused(lib, attend(lib, cache(page_size=1024), max_pages=1 << 21))           # slots of a sequence
    refused(lib, attend(lib, cache(n_pages=1 << 30, kv_heads=2)))                 # rows of pages and heads
    refused(lib, attend(lib, cache(), T=1024, heads=1 << 16))                     # drafted tokens times query heads
    refused(lib, attend(lib, cache(page_size=1024), B=65535, max_pages=1 << 12))  # tiles of all sequences, few rows
    refused(lib, attend(lib, cache(page_size=1024), B=65535, T=64, max_pages=1 << 14))


def test_cache_read_batch(lib):  # noqa: F811
    refused(lib, lib.fa_cache_read(ctypes.byref(cache()), 1, 65536, 4, P, 2, P, P, P, None))
