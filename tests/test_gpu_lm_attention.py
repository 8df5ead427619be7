"""Attention of drafted tokens over many sequences, tiles and cuts, against a plain 64-bit
implementation on the whole batch.  Tolerances are those of the model-side operators: with
ds = 2^-17 max_t scale sum_d |q_d k_d| and w = sum_t p |v|, a result is off by at most
(u + 4 ds) w, u = 2^-8 for bf16 weights and 2^-10 for fp16 ones, plus its own rounding."""
import pytest

torch = pytest.importorskip("torch")

import lm_reference as ref  # noqa: E402
from constrained_decoding_diffusion_gb300 import lm  # noqa: E402

pytestmark = pytest.mark.gpu

BF, HF, F8 = torch.bfloat16, torch.float16, torch.float8_e4m3fn


def make(seed, length, T, kv, page, dim, fmt, spread=0.0):
    """A filled cache whose sequences' pages lie in no order; e4m3 scales vary by 2^(+-spread)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    B, per = len(length), max(1, -(-(max(length) + T) // page))
    pages = B * per + 1
    table = torch.randperm(pages, generator=torch.Generator().manual_seed(seed))[:B * per].int().view(B, per).cuda()
    shape = (pages, kv, page, dim)
    k, v = (torch.randn(shape, generator=g, device="cuda") for _ in range(2))
    if fmt != F8:
        return lm.KVCache(k.to(fmt), v.to(fmt)), table
    ks, vs = (torch.exp2(spread * (2 * torch.rand(shape[:3], generator=g, device="cuda") - 1)) / 128 for _ in range(2))
    return lm.KVCache(*((100 * x).clamp(-448, 448).to(F8) for x in (k, v)), ks, vs), table


def plain(q, cache, table, length, seen, count, scale):
    """(out, lse, w, size); seen [B, T, T] says what of the draft a drafted token sees."""
    B, T, H, D = q.shape
    kv, page = cache.k.shape[1:3]
    n = table.shape[1] * page

    def rows(x, s):
        x = x.float().double()
        if s is not None:
            x = x * s.double()[..., None]
        return x[table.long()].permute(0, 2, 1, 3, 4).reshape(B, kv, n, D)
    k, v = rows(cache.k, cache.k_scale), rows(cache.v, cache.v_scale)
    qq = q.double().view(B, T, kv, H // kv, D).permute(0, 2, 1, 3, 4)
    s = scale * torch.einsum("bhtgd,bhnd->bhtgn", qq, k)
    size = scale * torch.einsum("bhtgd,bhnd->bhtgn", qq.abs(), k.abs())
    at = torch.arange(n, device="cuda")
    ok = (at[None, None] < length.view(B, 1, 1)).expand(B, T, n).clone()
    for b in range(B):
        n0, use = int(length[b]), int(count[b])
        ok[b, :, n0:n0 + T] |= seen[b] & (torch.arange(T, device="cuda") < use)
        ok[b, use:] = False
    s = s.masked_fill(~ok[:, None, :, None], -torch.inf)
    lse = torch.logsumexp(s, -1)
    p = torch.nan_to_num(torch.exp(s - lse[..., None]))
    size = size.masked_fill(~ok[:, None, :, None], 0).amax(-1)

    def back(x):
        return x.permute(0, 2, 1, 3, *range(4, x.dim())).reshape(B, T, H, *x.shape[4:])
    return [back(x) for x in (torch.einsum("bhtgn,bhnd->bhtgd", p, v), lse, torch.einsum("bhtgn,bhnd->bhtgd", p, v.abs()), size)]


def check(q, cache, table, length, seen=None, count=None, attend=None):
    B, T, H, D = q.shape
    length = torch.tensor(length, dtype=torch.int32).cuda()
    mask = None
    if seen is None:
        seen = torch.ones(B, T, T, dtype=torch.bool).tril().cuda()
        mask, _ = lm.fa_tree_mask(torch.arange(-1, T - 1, dtype=torch.int32).expand(B, T).contiguous().cuda())
    use = torch.full((B,), T, dtype=torch.int32, device="cuda") if count is None else torch.tensor(count, dtype=torch.int32).cuda()
    attend = attend or lm.TreeAttention(B, T, H, cache.k.shape[1], D, q.dtype)
    attend.out.fill_(9.0)
    attend.lse.fill_(9.0)
    out, lse = attend(q, cache, table, length, mask, None if count is None else use)
    want, wl, w, size = plain(q, cache, table, length, seen, use, D ** -0.5)
    assert torch.isfinite(want).all()
    ds = 2.0 ** -17 * size
    u = 2.0 ** -8 if cache.k.dtype == BF else 2.0 ** -10
    tol = (u + 4 * ds[..., None]) * w + ref.HALF_ULP[q.dtype] * want.abs() + ref.TINY[q.dtype]
    assert ((out.double() - want).abs() <= tol).all()
    assert torch.equal(torch.isneginf(lse), torch.isneginf(wl))
    some = ~torch.isneginf(wl)
    assert ((lse.double() - wl).abs()[some] <= (ds + 4e-6 * wl.abs().clamp_min(1))[some]).all()
    return out, lse


def queries(seed, *shape, dtype):
    return torch.randn(shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").to(dtype)


@pytest.mark.parametrize("fmt,dtype,dim,page", [(BF, BF, 128, 64), (HF, HF, 64, 16), (F8, BF, 128, 16), (F8, HF, 64, 64),
                                                (BF, BF, 80, 2), (F8, BF, 112, 128), (HF, HF, 48, 256)])
@pytest.mark.parametrize("T,group", [(1, 1), (1, 4), (2, 8), (16, 1), (17, 1), (40, 4)])
def test_long_contexts_in_many_tiles(fmt, dtype, dim, page, T, group):
    """Several tiles of several units in one run, so that every buffer is filled many times."""
    length = [3000, 1, 2049, 0, 700, 2999, 128, 1531]
    cache, table = make(T + dim, length, T, 8, page, dim, fmt, spread=3.0)
    q = queries(T, len(length), T, 8 * group, dim, dtype=dtype)
    first = [x.clone() for x in check(q, cache, table, length)]
    assert all(torch.equal(x, y) for x, y in zip(first, check(q, cache, table, length)))


@pytest.mark.parametrize("fmt,dtype", [(BF, BF), (F8, HF)])
@pytest.mark.parametrize("T,group", [(1, 2), (3, 4), (20, 1)])
def test_more_units_than_runs(fmt, dtype, T, group):
    """Hundreds of short sequences, some empty, with drafts of different lengths."""
    B = 333
    length = [(7 * b * b) % 150 if b % 5 else 0 for b in range(B)]
    count = [(b * 3) % (T + 1) for b in range(B)]
    cache, table = make(B, length, T, 4, 16, 64, fmt)
    check(queries(3, B, T, 4 * group, 64, dtype=dtype), cache, table, length, count=count)


@pytest.mark.parametrize("fmt,dtype", [(HF, HF), (F8, BF)])
@pytest.mark.parametrize("T,group", [(1, 1), (1, 4), (2, 1), (16, 1), (9, 2)])
def test_one_long_sequence_over_all_runs(fmt, dtype, T, group):
    """More partial results of a unit than lanes join them, and of one row to sixteen."""
    length = [41003]
    cache, table = make(T, length, T, 1, 64, 128, fmt, spread=6.0)
    check(queries(5, 1, T, group, 128, dtype=dtype), cache, table, length)


@pytest.mark.parametrize("T,group", [(1, 4), (24, 1)])
@pytest.mark.parametrize("scale", [0.0, 2.0 ** -100, 2.0 ** -60, 2.0 ** 60])
def test_values_of_any_magnitude(T, group, scale):
    """Vectors of zeros have the scale 0; nothing about the weights depends on the values."""
    length = [500, 90]
    cache, table = make(4, length, T, 2, 16, 128, F8)
    q = queries(4, 2, T, 2 * group, 128, dtype=BF)
    _, want = check(q, cache, table, length)
    want = want.clone()
    cache.v_scale.mul_(scale)
    _, lse = check(q, cache, table, length)
    assert (lse - want).abs().max() <= 8e-6 * want.abs().max()


@pytest.mark.parametrize("T", [1, 30])
def test_a_zero_query_weighs_all_alike(T):
    length = [300]
    cache, table = make(9, length, T, 1, 32, 64, F8, spread=4.0)
    q = torch.zeros(1, T, 2, 64, dtype=HF, device="cuda")
    _, lse = check(q, cache, table, length)
    seen = torch.arange(301, 301 + T, device="cuda").float().log()
    assert (lse[0, :, 0] - seen).abs().max() <= 4e-6 * 8
