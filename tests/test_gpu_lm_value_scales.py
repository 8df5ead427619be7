"""Value scales of an 8-bit cache that differ by many powers of two.  A weight is rounded to fp16 together with
its value's scale, relative to the largest such product that a row sees, so a large scale in a slot of little
weight takes no bits from the others.

Tolerance: that of the model-side operators with fp16 weights, (2^-10 + 4 ds) w + half a unit of the result, plus
what fp16's last step leaves of small products: half a step is 2^-25, the largest product is at least
2^3.5 of the same measure (it is aimed at 2^4 by whole powers of two), so at most 2^-28 max_t(p_t s_t) sum_t |code_t|.
Where a tile's scales are within 16 times one another the largest product may be as small as 2^-0.5; the tolerance
leaves that out."""
import pytest

torch = pytest.importorskip("torch")

import lm_reference as ref  # noqa: E402
from constrained_decoding_diffusion_gb300 import lm  # noqa: E402
from test_gpu_lm_attention import F8, make, plain, queries  # noqa: E402

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


def check(q, cache, table, length):
    B, T, H, D = q.shape
    n = torch.tensor(length, dtype=torch.int32).cuda()
    out, lse = lm.TreeAttention(B, T, H, cache.k.shape[1], D, q.dtype)(q, cache, table, n)
    seen, use = torch.ones(B, T, T, dtype=torch.bool, device="cuda"), torch.full((B,), T, dtype=torch.int32, device="cuda")
    want, wl, w, size = plain(q, cache, table, n, seen, use, D ** -0.5)
    # the largest product of a weight and a scale, and the sum of all codes' magnitudes
    slots, kv = table.shape[1] * cache.k.shape[2], cache.k.shape[1]
    scale = cache.v_scale.double()[table.long()].permute(0, 2, 1, 3).reshape(B, kv, slots)
    k = (cache.k.float().double() * cache.k_scale.double()[..., None])[table.long()].permute(0, 2, 1, 3, 4).reshape(B, kv, slots, D)
    code = cache.v.float().double().abs()[table.long()].permute(0, 2, 1, 3, 4).reshape(B, kv, slots, D)
    sees = (torch.arange(slots, device="cuda") < (n + T)[:, None])[:, None, None, None]
    s = torch.einsum("bthgd,bhnd->bthgn", q.double().view(B, T, kv, H // kv, D), k) * D ** -0.5
    p = torch.exp(s - wl.view(B, T, kv, H // kv, 1)).masked_fill(~sees, 0)
    most = (p * scale[:, None, :, None]).amax(-1).view(B, T, H)
    codes = (code * sees[:, :, 0, 0, :, None]).sum(2).repeat_interleave(H // kv, 1)[:, None]
    ds = 2.0 ** -17 * size
    tol = (2.0 ** -10 + 4 * ds[..., None]) * w + 2.0 ** -28 * most[..., None] * codes + ref.HALF_ULP[q.dtype] * want.abs() + ref.TINY[q.dtype]
    assert torch.isfinite(want).all()
    assert ((out.double() - want).abs() <= tol).all(), float(((out.double() - want).abs() / tol).max())
    assert ((lse.double() - wl).abs() <= ds + 4e-6 * wl.abs().clamp_min(1)).all()


@pytest.mark.parametrize("dtype,dim", [(BF, 64), (HF, 128)])
@pytest.mark.parametrize("T,group", [(1, 1), (1, 12), (18, 1), (12, 4), (100, 1), (200, 1)])
@pytest.mark.parametrize("power", [16, 22, 30, 60])
@pytest.mark.parametrize("where", [5, 700, 1499])
def test_a_large_scale_where_the_weight_is_small(dtype, dim, T, group, power, where):
    """One slot with the scale 2^power times the others' and a score some fifty bits below theirs."""
    length = [1500]
    cache, table = make(T + group, length, T, 1, 16, dim, F8)
    q = queries(1, 1, 1, 1, dim, dtype=dtype) + 0.05 * queries(2, 1, T, group, dim, dtype=dtype)
    q = q.to(dtype)
    p, g = int(table[0, where // 16]), where % 16
    cache.k[p, 0, g] = (-448 * q[0, 0, 0].float().sign()).to(F8)
    cache.k_scale[p, 0, g] *= 4
    cache.v_scale[p, 0, g] *= 2.0 ** power
    check(q, cache, table, length)


@pytest.mark.parametrize("T,group", [(1, 4), (3, 5), (20, 1), (24, 4), (50, 4)])
@pytest.mark.parametrize("spread", [9.0, 18.0, 36.0])
def test_scales_of_any_spread(T, group, spread):
    length = [2100, 130, 3, 900]
    cache, table = make(T, length, T, 2, 32, 128, F8, spread=spread)
    check(2 * queries(3, 4, T, 2 * group, 128, dtype=BF), cache, table, length)


@pytest.mark.parametrize("T,group", [(1, 4), (20, 1), (40, 4)])
def test_scales_against_scores(T, group):
    """Scores that rise by hundreds along the context while the scales fall, and the other way round: the
    products stay level or move by twice as much."""
    for sign in (1.0, -1.0):
        length = [1000]
        cache, table = make(T, length, T, 1, 16, 64, F8)
        q = queries(4, 1, 1, 1, 64, dtype=BF).abs() + 0.05 * queries(5, 1, T, group, 64, dtype=BF)
        q = q.to(BF)
        at = torch.arange(1000 + T, device="cuda")
        p, g = table[0, at // 16].long(), at % 16
        rise = at / (1000.0 + T)
        cache.k[p, 0, g] = cache.k[p, 0, g].float().abs().to(F8)
        cache.k_scale[p, 0, g] *= 1 + 3 * rise
        cache.v_scale[p, 0, g] *= torch.exp2(-sign * 60 * rise)
        check(q, cache, table, length)
