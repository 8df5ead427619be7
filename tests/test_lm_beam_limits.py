"""Beams and vocabularies at the end of 32-bit indices, refused before any CUDA call (CPU only; the pointers
are never followed)."""
import ctypes

import pytest

from constrained_decoding_diffusion_gb300 import native
from test_lm_refusals import P, lib, refused  # noqa: F401


@pytest.mark.parametrize("K,V", [(1, 2 ** 31 - 1), (1, 2 ** 31 - 8192), (1, 2 ** 31 - 2 ** 14), (2 ** 31 - 1, 1), (2 ** 31 - 600, 1)])
def test_indices_of_cells_and_batches(lib, K, V):  # noqa: F811
    n = ctypes.c_size_t()
    refused(lib, lib.fa_beam_select_workspace_bytes(1, K, V, 4, ctypes.byref(n)))
    out = [P + (i + 8 << 40) for i in range(6)]
    refused(lib, lib.fa_beam_select(0, 1, K, V, 4, P, V, V, out[0], None, 0, None, None, out[1], out[2], out[3], None, P, 1 << 40, None))


@pytest.mark.parametrize("K,V", [(1, 2 ** 31 - 2 ** 14 - 1), (2 ** 31 - 2 ** 14 - 1, 1), (46340, 46340)])
def test_just_below(lib, K, V):  # noqa: F811
    n = ctypes.c_size_t()
    assert lib.fa_beam_select_workspace_bytes(1, K, V, 256, ctypes.byref(n)) == native.FA_OK
    assert n.value == 8 * 256 * 608
