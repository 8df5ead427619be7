"""Latent attention of more units (sequences, and blocks of 64 rows of them) than the GPU has SMs, up to the most sequences."""
import pytest

torch = pytest.importorskip("torch")

from constrained_decoding_diffusion_gb300 import lm, native  # noqa: E402
from test_gpu_latent import BF, HF, chains, check, ints, make, normal  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,latent,rope,T,H", [(BF, 512, 64, 1, 16), (HF, 128, 16, 2, 40), (BF, 256, 32, 3, 64)])
@pytest.mark.parametrize("length", [[(53 * b) % 211 for b in range(300)],
                                    [0] * 100 + [30000] + [1] * 100 + [700, 64, 63, 65] * 10,
                                    [(53 * b) % 211 for b in range(520)],
                                    [20000, 0, 9000] + [3] * 600])
def test_units_cut_by_runs(length, dtype, latent, rope, T, H):
    """Short ones that are not cut, units cut once, and a unit cut into very many parts."""
    cache, table = make(len(length), length, T, 16, latent, rope, dtype)
    check(normal(T, len(length), T, H, latent + rope, dtype=dtype), cache, table, length, 0.07, chains(len(length), T))


@pytest.mark.parametrize("T,H,length", [(1, 16, [(37 * b) % 300 for b in range(700)]), (2, 40, [100] * 300 + [50000] + [64] * 300)])
def test_a_wait_that_runs_out_among_many_sequences(T, H, length):
    """The rows that the first block has a part in are NaN, whole units and a cut one's; all others are right."""
    B = len(length)
    cache, table = make(T, length, T, 16, 128, 16, BF)
    q, n = normal(H, B, T, H, 144, dtype=BF), ints(length)
    attend = lm.LatentAttention(B, T, H, 128, 16, BF)
    clean, lse = (x.clone() for x in attend(q, cache, table, n, 0.07))
    native.fa_debug_inject_wait_timeouts(1)
    try:
        out, l2 = (x.clone() for x in attend(q, cache, table, n, 0.07))
    finally:
        native.fa_debug_inject_wait_timeouts(0)
    lost = torch.isnan(l2)
    assert torch.equal(lost, torch.isnan(out).all(-1)) and torch.equal(lost, torch.isnan(out).any(-1))
    assert torch.equal(out[~lost], clean[~lost]) and torch.equal(l2[~lost], lse[~lost])
    units = [rows for b in range(B) for rows in lost.view(B, T * H)[b].split(64)]
    first = sum(bool(x.any()) for x in units)
    assert 1 <= first < len(units) and all(bool(x.all()) for x in units[:first])
    again, l3 = attend(q, cache, table, n, 0.07)
    assert torch.equal(again, clean) and torch.equal(l3, lse)


def test_time_does_not_grow_with_the_square_of_the_sequences():
    """Four times the sequences take less than eight times as long (fourteen with a plan by every sequence)."""
    times = []
    for B in (16384, 65535):
        cache = lm.LatentCache(torch.zeros(B, 64, 144, dtype=BF, device="cuda"), 128)
        table = torch.arange(B, dtype=torch.int32, device="cuda").view(B, 1)
        q = normal(1, B, 1, 16, 144, dtype=BF)
        attend, length = lm.LatentAttention(B, 1, 16, 128, 16, BF), ints([63] * B)
        start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        took = []
        for _ in range(4):
            start.record()
            attend(q, cache, table, length, 0.1)
            end.record()
            end.synchronize()
            took.append(start.elapsed_time(end))
        times.append(min(took))
    assert times[1] < 8 * times[0], times
