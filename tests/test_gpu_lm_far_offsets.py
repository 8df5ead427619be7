"""Offsets past 32 bits: pages, queries, rows and cells that lie more than 4 GB behind their base give the bits
that the same data give near it."""
import pytest

torch = pytest.importorskip("torch")

from constrained_decoding_diffusion_gb300 import lm  # noqa: E402
from test_gpu_lm_attention import F8, queries  # noqa: E402

pytestmark = pytest.mark.gpu

BF, HF, FP = torch.bfloat16, torch.float16, torch.float32


def pair(fmt, dim, page, kv, per, B):
    """A small cache with a table, and the same pages at the far end of a cache of more than 5 GB a side."""
    size = kv * page * dim * (1 if fmt == F8 else 2)
    n_far = int(5.2e9) // size
    near, far = lm.KVCache.empty(B * per, kv, page, dim, fmt), lm.KVCache.empty(n_far, kv, page, dim, fmt)
    table = torch.randperm(B * per, generator=torch.Generator().manual_seed(1)).int().view(B, per).cuda()
    return near, far, table, table + (n_far - B * per)


def tail(far, near):
    return [None if x is None else x[-y.shape[0]:] for x, y in zip(far, near)]


def same(far, near):
    return all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(tail(far, near), near) if x is not None)


@pytest.mark.parametrize("fmt,dtype", [(BF, BF), (F8, BF)])
@pytest.mark.parametrize("dim,page", [(128, 64), (64, 4)])
def test_cache_and_attention(fmt, dtype, dim, page):
    B, kv, T = 2, 4, 300
    near, far, t_near, t_far = pair(fmt, dim, page, kv, -(-400 // page), B)
    for x, y in zip(near, tail(far, near)):
        if x is not None:
            x.view(torch.uint8).zero_()
            y.view(torch.uint8).zero_()
    k, v = queries(1, B, T, kv, dim, dtype=dtype), queries(2, B, T, kv, dim, dtype=dtype)
    start = torch.tensor([3, 50], dtype=torch.int32).cuda()
    pos = torch.arange(T, dtype=torch.int32, device="cuda").expand(B, T).contiguous()
    phase, _ = lm.rope_phases(dim)
    for cache, table in ((near, t_near), (far, t_far)):
        lm.fa_cache_write(cache, k, v, table, start, positions=pos, phase=phase)
    assert same(far, near)
    path = torch.tensor([[0, 4, 5, 90], [2, 3, 77, -1]], dtype=torch.int32).cuda()
    out = []
    for cache, table in ((near, t_near), (far, t_far)):
        lm.fa_cache_keep(cache, table, start + 100, path)
        got = [torch.empty((B, 320, kv, dim), dtype=dtype, device="cuda") for _ in range(2)]
        lm.fa_cache_read(cache, table, start + T, *got)
        for T2, group in ((1, 4), (3, 5), (16, 4), (50, 2), (60, 4)):
            q = queries(T2, B, T2, kv * group, dim, dtype=dtype)
            got += [x.clone() for x in lm.TreeAttention(B, T2, kv * group, kv, dim, dtype)(q, cache, table, start + T - T2)]
        out.append(got)
    assert same(far, near)
    assert all(torch.equal(x, y) and x.float().abs().sum() > 0 for x, y in zip(*out))


@pytest.mark.parametrize("rot,shift", [(128, 0), (96, 0), (96, 1)])
def test_positions_of_many_elements(rot, shift):
    """2^31 elements and more; shift: rows that are not aligned."""
    n, heads, dim = 270001, 64, 128 + 8 * shift
    x = torch.empty((n, heads, dim), dtype=BF, device="cuda")[..., shift:shift + 128]
    assert x[-1].storage_offset() > 2 ** 31
    end = queries(1, 1000, heads, 128, dtype=BF)
    x[-1000:] = end
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    phase, _ = lm.rope_phases(rot)
    lm.fa_rope(x, pos, phase, out=x)
    assert torch.equal(x[-1000:], lm.fa_rope(end, pos[-1000:], phase))


@pytest.mark.parametrize("dtype", [BF, FP])
def test_beams_of_many_cells(dtype):
    N, K, V, top = 150, 16, 1000003, 20
    g = torch.Generator(device="cuda").manual_seed(1)
    logp = torch.full((N, K, V), -9.0, dtype=dtype, device="cuda")
    logp[-2:, :, ::50] = torch.randn((2, K, (V + 49) // 50), generator=g, device="cuda").to(dtype)
    assert logp.numel() > 2 ** 31
    scores = torch.randn((N, K), generator=g, device="cuda")
    got = lm.BeamSelect(N, K, V, top, dtype)(logp, scores)
    want = lm.BeamSelect(2, K, V, top, dtype)(logp[-2:].clone(), scores[-2:].contiguous())
    for x, y in zip(got[:3], want[:3]):
        assert torch.equal(x[-2:], y)
