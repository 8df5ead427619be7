"""Attention of drafted tokens when drafted values are not finite.  Rows that do not see them keep
their very bits; rows that do come out with NaN or the infinity in the columns that hold it."""
import pytest

torch = pytest.importorskip("torch")

from constrained_decoding_diffusion_gb300 import lm  # noqa: E402
from test_gpu_lm_attention import F8, make, queries  # noqa: E402

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


def chain(B, T):
    mask, _ = lm.fa_tree_mask(torch.arange(-1, T - 1, dtype=torch.int32).expand(B, T).contiguous().cuda())
    return mask


def put(x, table, at, value):
    """x[page, :, place, ...] of slot at[b] of every sequence b (none where at[b] < 0) becomes value."""
    page = x.shape[2]
    b = (at >= 0).nonzero()[:, 0]
    p = table[b, (at[b] // page).long()].long()
    x[p, :, (at[b] % page).long()] = value


@pytest.mark.parametrize("dtype,dim", [(BF, 64), (HF, 128)])
def test_marked_scales_behind_runs_of_short_sequences(dtype, dim):
    """Many sequences of one tile before one of two, whose drafted slots lie in the second: the stream
    that has only the second tile comes to it long before the other stream."""
    B, T = 3000, 20
    length = [150 + b % 80 if b % 11 == 10 else (37 * b) % 109 for b in range(B)]
    cache, table = make(B, length, T, 1, 16, dim, F8)
    q, n, mask = queries(1, B, T, 1, dim, dtype=dtype), torch.tensor(length, dtype=torch.int32).cuda(), chain(B, T)
    attend = lm.TreeAttention(B, T, 1, 1, dim, dtype)
    clean, lse = (x.clone() for x in attend(q, cache, table, n, mask))
    bad = torch.where(n >= 150, 3, -1)
    put(cache.v_scale, table, torch.where(bad >= 0, n + 3, -1), float("nan"))
    sees = (torch.arange(T, device="cuda") >= 3) & (bad >= 0)[:, None]
    for _ in range(5):
        out, l2 = attend(q, cache, table, n, mask)
        assert torch.isnan(out[sees]).all() and torch.isfinite(l2[sees]).all()
        assert torch.equal(out[~sees], clean[~sees]) and torch.equal(l2[~sees], lse[~sees])
