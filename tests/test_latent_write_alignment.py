"""fa_latent_write refuses inputs between two elements before any CUDA call (CPU only; the pointers are never followed)."""
import ctypes

import pytest

from test_serving_refusals import P, lib, latent, refused, write  # noqa: F401


@pytest.mark.parametrize("dtype,off", [(0, 1), (0, 2), (0, 3), (1, 1), (2, 1), (2, 3)])
@pytest.mark.parametrize("name", ["x", "key"])
def test_inputs_between_elements(lib, name, dtype, off):  # noqa: F811
    refused(lib, write(lib, ctypes.byref(latent()), dtype=dtype, **{name: P + off}))
    assert b"aligned" in lib.fa_last_error()
