"""Values that are not finite, in every form of the attention kernels: up to 8 and up to 16 rows without
shared tiles; four, two and one copies of the rows, two row tiles and two row blocks on the tensor cores; contexts
of one tile, of several and long enough to be cut.

Only one drafted token sees the odd slot.  The other rows keep their very bits.  In the row that sees it a
value changes the columns that hold it and no others, since columns of a product are worked out apart."""
import math

import pytest

torch = pytest.importorskip("torch")

from constrained_decoding_diffusion_gb300 import lm  # noqa: E402
from test_gpu_lm_attention import F8, make, queries  # noqa: E402

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16
LENGTH = [5, 300, 5000, 0, 126]


@pytest.mark.parametrize("T,group", [(3, 1), (3, 4), (18, 1), (12, 4), (25, 4), (50, 4), (100, 4)])
@pytest.mark.parametrize("fmt,dtype,dim", [(BF, BF, 128), (HF, HF, 64), (F8, BF, 64), (F8, HF, 128), (BF, BF, 80)])
def test_who_sees_what(T, group, fmt, dtype, dim):
    B, kv, col = len(LENGTH), 2, 5
    cache, table = make(T + dim, LENGTH, T, kv, 16, dim, fmt)
    q = queries(T, B, T, kv * group, dim, dtype=dtype)
    n = torch.tensor(LENGTH, dtype=torch.int32).cuda()
    parents = torch.arange(-1, T - 1, dtype=torch.int32)
    parents[1:] = 0                                    # leaves, so that each is seen by itself
    mask, _ = lm.fa_tree_mask(parents.expand(B, T).contiguous().cuda())
    attend = lm.TreeAttention(B, T, kv * group, kv, dim, dtype)
    clean, lse = (x.clone() for x in attend(q, cache, table, n, mask))
    assert torch.isfinite(clean).all() and torch.isfinite(lse).all()
    for t in sorted({1, 2, T - 1}):
        at = n + t
        page, place = table[torch.arange(B, device="cuda"), (at // 16).long()].long(), (at % 16).long()
        others = torch.arange(T, device="cuda") != t
        rest = torch.arange(dim, device="cuda") != col

        def run():
            out, l2 = attend(q, cache, table, n, mask)
            assert torch.equal(out[:, others], clean[:, others]) and torch.equal(l2[:, others], lse[:, others])
            return out[:, t], l2[:, t]

        if fmt == F8:
            codes = cache.v.view(torch.uint8)
            kept = codes[page, :, place, col].clone()
            codes[page, :, place, col] = 0x7F
            out, l2 = run()
            assert torch.isnan(out[..., col]).all() and torch.equal(out[..., rest], clean[:, t][..., rest])
            assert torch.equal(l2, lse[:, t])
            codes[page, :, place, col] = kept
            for x, bad in ((cache.v_scale, math.nan), (cache.v_scale, math.inf), (cache.k_scale, math.nan)):
                kept = x[page, :, place].clone()
                x[page, :, place] = bad
                out, l2 = run()
                assert torch.isnan(out).all()
                if x is cache.v_scale:
                    assert ((l2 - lse[:, t]).abs() <= 8e-6 * lse[:, t].abs().clamp_min(1)).all()
                else:
                    assert torch.isnan(l2).all()
                x[page, :, place] = kept
        else:
            for bad in (math.nan, math.inf, -math.inf):
                kept = cache.v[page, :, place, col].clone()
                cache.v[page, :, place, col] = bad
                out, l2 = run()
                want = torch.full_like(out[..., col], bad)
                assert torch.equal(torch.nan_to_num(out[..., col], 7.0, 8.0, -8.0), torch.nan_to_num(want, 7.0, 8.0, -8.0))
                assert torch.equal(out[..., rest], clean[:, t][..., rest]) and torch.equal(l2, lse[:, t])
                cache.v[page, :, place, col] = kept
                kept = cache.k[page, :, place, col].clone()
                cache.k[page, :, place, col] = bad
                out, l2 = run()
                if math.isnan(bad):
                    assert torch.isnan(out).all() and torch.isnan(l2).all()
                cache.k[page, :, place, col] = kept
    out, l2 = attend(q, cache, table, n, mask)
    assert torch.equal(out, clean) and torch.equal(l2, lse)


@pytest.mark.parametrize("T,group", [(1, 1), (1, 12), (18, 1), (12, 4), (25, 4), (50, 4)])
@pytest.mark.parametrize("fmt,dtype,dim", [(BF, BF, 128), (HF, HF, 64), (F8, BF, 64), (F8, HF, 128)])
def test_before_the_draft(T, group, fmt, dtype, dim):
    """A value that is not finite before the draft is seen by all rows of its sequence and head and by no others."""
    B, kv, col = 4, 2, 7
    length = [700, 90, 5000, 300]
    cache, table = make(T + dim, length, T, kv, 16, dim, fmt)
    q = queries(T, B, T, kv * group, dim, dtype=dtype)
    n = torch.tensor(length, dtype=torch.int32).cuda()
    attend = lm.TreeAttention(B, T, kv * group, kv, dim, dtype)
    clean, lse = (x.clone() for x in attend(q, cache, table, n))
    for slot in (0, 77, 699):
        p, g = int(table[0, slot // 16]), slot % 16
        x = cache.v.view(torch.uint8) if fmt == F8 else cache.v
        kept = x[p, 1, g, col].clone()
        for bad in ([0x7F] if fmt == F8 else [math.nan, math.inf, -math.inf]):
            x[p, 1, g, col] = bad
            out, l2 = attend(q, cache, table, n)
            assert torch.equal(l2, lse)
            assert torch.equal(out[1:], clean[1:]) and torch.equal(out[0, :, :group], clean[0, :, :group])
            got = out[0, :, group:]
            assert not torch.isfinite(got[..., col]).any()
            rest = torch.arange(dim, device="cuda") != col
            assert torch.equal(got[..., rest], clean[0, :, group:][..., rest])
        x[p, 1, g, col] = kept
