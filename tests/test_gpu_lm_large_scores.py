"""Scores so large that their differences from the row's largest are what is left of fp32: the largest still
takes all the weight, equal ones share it, and nothing overflows or vanishes.

Tolerance: the weights are one or nothing here (scores differ by a twentieth of themselves, hundreds at least), so a
result is the winner's value up to the weight's rounding, u = 2^-8 in bf16 and 2^-10 in fp16, and its own."""
import pytest

torch = pytest.importorskip("torch")

import lm_reference as ref  # noqa: E402
from constrained_decoding_diffusion_gb300 import lm  # noqa: E402
from test_gpu_lm_attention import F8, make, queries  # noqa: E402

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16
ROWS = [(1, 1), (1, 12), (18, 1), (12, 4), (100, 1), (200, 1)]


def signs(dim):
    return torch.randn(dim, generator=torch.Generator().manual_seed(1)).sign().cuda()


def fill(cache, table, n, along, dim):
    """Keys along[t] times a vector of signs in the slots t < n of every head of sequence 0, with scales of one."""
    t = torch.arange(n, device="cuda")
    page = cache.k.shape[2]
    cache.k[table[0, t // page].long(), :, t % page] = (along.cuda()[:, None] * signs(dim))[:, None].to(cache.k.dtype)
    if cache.k_scale is not None:
        cache.k_scale.fill_(1.0)


def run(cache, table, n, T, group, dim, dtype, power):
    """The queries 2^power (1, 2 or 3) times the signs, and what comes of them."""
    kv = cache.k.shape[1]
    rows = (torch.arange(T * group * kv, device="cuda") % 3 + 1).view(1, T, group * kv, 1)
    q = (2.0 ** power * rows * signs(dim)).to(dtype)
    length = torch.tensor([n - T], dtype=torch.int32).cuda()
    attend = lm.TreeAttention(1, T, kv * group, kv, dim, dtype)
    attend.out.fill_(9.0)
    out, lse = attend(q, cache, table, length)
    return out.double(), lse.double(), rows.double()[..., 0] * 2.0 ** power * dim ** 0.5


def values(cache, table, n):
    """[n, heads, dim] in 64 bits."""
    t = torch.arange(n, device="cuda")
    page = cache.k.shape[2]
    at = table[0, t // page].long(), slice(None), t % page
    v = cache.v[at].float().double()
    return v if cache.v_scale is None else v * cache.v_scale[at].double()[..., None]


@pytest.mark.parametrize("fmt,dtype,power", [(BF, BF, p) for p in (14, 20, 24, 32, 60)] + [(HF, HF, 13)] +
                         [(F8, BF, p) for p in (14, 20, 24, 32, 60)] + [(F8, HF, 13)])
@pytest.mark.parametrize("T,group", ROWS)
@pytest.mark.parametrize("sign", [1, -1])
def test_the_largest_takes_all(fmt, dtype, power, T, group, sign):
    dim = 128 if T in (18, 100) or group == 12 else 64
    for n, winner in ((T + 3, 1), (700, 2), (700, 350), (700, 699), (1500, 1100)):
        cache, table = make(7, [n - T], T, 2, 16, dim, fmt)
        along = 1.0 + torch.randint(0, 7, (n,), generator=torch.Generator().manual_seed(n)) / 8
        along[winner] = 2.0
        if sign < 0:
            along = along - 3.0
        # fp16 keys of 256 (exact) reach what bf16 queries reach alone
        stretch = 256.0 if fmt == HF else 1.0
        fill(cache, table, n, along * stretch, dim)
        out, lse, size = run(cache, table, n, T, group, dim, dtype, power)
        want = values(cache, table, n)[winner].repeat_interleave(group, 0)[None, None]
        u = 2.0 ** -8 if fmt == BF else 2.0 ** -10
        tol = (u + ref.HALF_ULP[dtype]) * want.abs() + ref.TINY[dtype]
        if fmt == F8:
            tol = tol + 2.0 ** -28 * 448 * cache.v_scale.max()      # fp16's last step against the largest weight
        assert ((out - want).abs() <= tol).all(), (n, winner, out[0, 0, 0, :4], want[0, 0, 0, :4])
        top = size * stretch * float(along[winner])
        assert ((lse - top).abs() <= 2.0 ** -17 * top.abs() + 4e-6 * top.abs()).all()


@pytest.mark.parametrize("fmt,dtype,power", [(BF, BF, 20), (BF, BF, 33), (BF, BF, 60), (F8, BF, 33), (F8, BF, 60)])
@pytest.mark.parametrize("T,group", ROWS)
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_equal_ones_share(fmt, dtype, power, T, group, sign):
    """All in one tile, so that no parts are joined by their logarithms."""
    n = 16 if T * group <= 16 else T + 20
    if n > 128:
        n = T
    cache, table = make(8, [n - T], T, 1, 16, 64, fmt)
    if cache.v_scale is not None:
        cache.v_scale.fill_(1.0)
    fill(cache, table, n, torch.full((n,), sign), 64)
    out, lse, size = run(cache, table, n, T, group, 64, dtype, power)
    v = values(cache, table, n)
    want, w = v.mean(0), v.abs().mean(0)
    if n <= 128:
        tol = 2.0 ** -8 * w + ref.HALF_ULP[dtype] * want.abs() + ref.TINY[dtype]
        assert ((out - want).abs() <= tol).all()
    assert torch.isfinite(out).all() and ((lse - sign * size).abs() <= 1e-5 * size).all()
