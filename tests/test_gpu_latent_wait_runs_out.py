"""A wait inside the latent attention that runs out: the rows its block has a part in come out as NaN, all others are
right, and the next call is unaffected."""
import pytest

torch = pytest.importorskip("torch")

from constrained_decoding_diffusion_gb300 import lm, native  # noqa: E402
from test_gpu_latent import BF, HF, ints, make, normal  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,size,latent,rope", [(BF, 64, 512, 64), (BF, 4, 128, 16), (HF, 16, 256, 32)])
@pytest.mark.parametrize("T,H", [(1, 16), (3, 40)])
@pytest.mark.parametrize("length", [[2000] * 9, [(37 * b) % 300 for b in range(400)]])
def test_rows_of_the_first_block(dtype, size, latent, rope, T, H, length):
    B = len(length)
    cache, table = make(T, length, T, size, latent, rope, dtype)
    q = normal(H, B, T, H, latent + rope, dtype=dtype)
    n = ints(length)
    attend = lm.LatentAttention(B, T, H, latent, rope, dtype)
    clean, lse = (x.clone() for x in attend(q, cache, table, n, 0.07))
    assert torch.isfinite(clean).all()
    native.fa_debug_inject_wait_timeouts(1)
    try:
        out, l2 = (x.clone() for x in attend(q, cache, table, n, 0.07))
    finally:
        native.fa_debug_inject_wait_timeouts(0)
    lost = torch.isnan(l2)
    assert torch.equal(lost, torch.isnan(out).all(-1)) and torch.equal(lost, torch.isnan(out).any(-1))
    assert torch.equal(out[~lost], clean[~lost]) and torch.equal(l2[~lost], lse[~lost])
    # the block takes the first units of the list: sequences, and blocks of 64 rows of them
    units = [rows for b in range(B) for rows in lost.view(B, T * H)[b].split(64)]
    some = [bool(x.any()) for x in units]
    first = sum(some)
    assert 1 <= first < len(units) and all(some[:first]) and all(bool(x.all()) for x in units[:first])
    out, l2 = attend(q, cache, table, n, 0.07)
    assert torch.equal(out, clean) and torch.equal(l2, lse)
