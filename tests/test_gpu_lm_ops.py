"""The model-side operators against plain 64-bit implementations: rotary positions, the paged
cache, attention of drafted tokens, beam selection.

Tolerances.  A stored result may be off by its type's rounding (half a unit in the last place)
plus the fp32 arithmetic before it.  Rotation: the angle is exact to 2^-24 of half a turn, sine
and cosine and the two products add a few units of 2^-24, so 1e-6 (|x0| + |x1|) mscale covers
them.  Attention: a score of 128 products summed in fp32 is off by at most 2^-17 of the sum of
their magnitudes, which scales its weight; each weight is rounded to 8 (bf16) or 11 bits for
the product with the values, so with w = sum p |v| the result is off by at most
(u + 4 ds) w, u = 2^-8 or 2^-10.  Beams: one fp32 addition, so everything is equal.
"""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import lm_reference as ref  # noqa: E402
from constrained_decoding_diffusion_gb300 import lm, native, synth  # noqa: E402

pytestmark = pytest.mark.gpu

BF, HF, FP, F8 = torch.bfloat16, torch.float16, torch.float32, torch.float8_e4m3fn


def gen(seed):
    return torch.Generator().manual_seed(seed)


def randn(seed, *shape, dtype=FP, scale=1.0):
    return (scale * torch.randn(shape, generator=gen(seed))).to(dtype).cuda()


def i32(x):
    return torch.as_tensor(x, dtype=torch.int32).cuda()


# ------------------------------------------------------------------ rotary positions

@pytest.mark.parametrize("dtype", [FP, HF, BF])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("n,heads,dim,rot", [(1, 1, 2, 2), (5, 3, 64, 64), (7, 2, 96, 32), (33, 5, 128, 64), (2, 40, 128, 128),
                                             (3, 1, 70, 26), (300, 4, 64, 0), (0, 4, 64, 64)])
def test_rope(dtype, interleaved, n, heads, dim, rot):
    x = randn(n + rot, n, heads, dim, dtype=dtype)
    pos = torch.randint(0, 100000, (n,), generator=gen(1)).int()
    if n > 2:
        pos[:3] = torch.tensor([0, 2 ** 31 - 1, -12345])
    phase, m = lm.rope_phases(rot)
    for inverse in (False, True):
        y = lm.fa_rope(x, pos.cuda(), phase, interleaved=interleaved, mscale=1.5 * m, inverse=inverse)
        want = ref.rope(x, pos, rot, interleaved=interleaved, mscale=1.5, inverse=inverse)
        tol = 1.5e-6 * ref.pair_sum(x, rot, interleaved) + ref.HALF_ULP[dtype] * np.abs(want) + ref.TINY[dtype]
        got = y.double().cpu().numpy()
        assert (np.abs(got - want) <= tol).all(), np.max(np.abs(got - want) - tol)
        assert torch.equal(y[:, :, rot:], x[:, :, rot:])


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("pad", [0, 3, 8])
def test_rope_strides_and_in_place(interleaved, pad):
    wide = randn(5, 6, 9, 64 + pad, dtype=BF)
    x = wide[:, 2:7, pad:]                           # strided, and with pad = 3 not 16-byte aligned
    pos = i32([3, 1, 4, 1, 5, 9])
    phase, _ = lm.rope_phases(48)
    want = lm.fa_rope(x.contiguous(), pos, phase, interleaved=interleaved)
    before = wide.clone()
    assert torch.equal(lm.fa_rope(x, pos, phase, interleaved=interleaved), want)
    assert torch.equal(wide, before)
    lm.fa_rope(x, pos, phase, out=x, interleaved=interleaved)
    assert torch.equal(x, want)
    before[:, 2:7, pad:] = want
    assert torch.equal(wide, before)                 # nothing beside it was written


@pytest.mark.parametrize("scaling,divide", [("linear", 4.0), ("base", None), ("blend", None)])
def test_rope_scaling(scaling, divide):
    phase, m = lm.rope_phases(64, scaling=scaling, factor=4.0, original_length=2048)
    turns = phase.cpu().numpy().astype(np.uint64).astype(np.float64) / 2.0 ** 64 * 2 * math.pi
    plain = 10000.0 ** (-np.arange(32) / 32.0)
    if scaling == "linear":
        want = plain / divide
    elif scaling == "base":
        want = (10000.0 * 4.0 ** (64 / 62)) ** (-np.arange(32) / 32.0)
        assert abs(want[-1] - plain[-1] / 4.0) < 1e-12 and want[0] == 1.0
    else:
        made = plain * 2048 / (2 * math.pi)
        keep = np.clip((made - 1.0) / 31.0, 0.0, 1.0)
        want = keep * plain + (1 - keep) * plain / 4.0
        assert abs(m - (0.1 * math.log(4.0) + 1.0)) < 1e-15
    np.testing.assert_allclose(turns, want, rtol=1e-13)


def test_rope_gradient():
    """The gradient is the transposed rotation: against the formula and against differences."""
    x = randn(3, 4, 2, 32).requires_grad_(True)
    g = randn(4, 4, 2, 32)
    pos = i32([0, 7, 1000, 77777])
    phase, _ = lm.rope_phases(16)
    y = lm.Rope.apply(x, pos, phase, True, 1.25)
    (y * g).sum().backward()
    want = ref.rope(g, pos, 16, interleaved=True, mscale=1.25, inverse=True)
    np.testing.assert_allclose(x.grad.double().cpu().numpy(), want, rtol=0, atol=1e-5)
    with torch.no_grad():
        for at in [(0, 0, 0), (1, 1, 5), (2, 0, 14), (3, 1, 15), (3, 0, 31)]:
            up, down = x.detach().clone(), x.detach().clone()
            up[at] += 1.0
            down[at] -= 1.0
            diff = ((lm.fa_rope(up, pos, phase, interleaved=True, mscale=1.25).double() -
                     lm.fa_rope(down, pos, phase, interleaved=True, mscale=1.25).double()) * g.double()).sum() / 2
            assert abs(float(diff) - float(x.grad[at])) < 2e-5     # linear: only rounding is left
    y = lm.Rope.apply(x, pos, phase)
    y.sum().backward()                                             # a broadcast gradient


# ------------------------------------------------------------------ the cache

def make_cache(seed, B, slots, heads, page, dim, dtype, spare=2, scale=1.0):
    """A cache filled with values, and a page table in no order."""
    per = max(1, -(-slots // page))
    pages = B * per + spare
    table = torch.randperm(pages, generator=gen(seed))[:B * per].int().view(B, per)
    shape = (pages, heads, page, dim)
    k, v = (scale * torch.randn(shape, generator=gen(seed + i)) for i in (1, 2))
    if dtype != F8:
        return lm.KVCache(k.to(dtype).cuda(), v.to(dtype).cuda()), table.cuda()
    ks, vs = (x.abs().amax(-1) / 448.0 for x in (k, v))
    return lm.KVCache((k / ks[..., None]).to(F8).cuda(), (v / vs[..., None]).to(F8).cuda(), ks.cuda(), vs.cuda()), table.cuda()


@pytest.mark.parametrize("fmt", [HF, BF, F8])
@pytest.mark.parametrize("dtype", [FP, HF, BF])
@pytest.mark.parametrize("page,dim,heads", [(1, 16, 1), (16, 64, 3), (64, 128, 2), (8, 80, 5), (128, 256, 1)])
def test_cache_write_and_read(fmt, dtype, page, dim, heads):
    B, T = 3, 21
    cache = lm.KVCache.empty(3 * (64 // page + 1), heads, page, dim, fmt)
    for x in cache:
        if x is not None:
            x.view(torch.uint8).fill_(0x37)
    before = [None if x is None else x.clone() for x in cache]
    per = cache.k.shape[0] // 3
    table = torch.randperm(3 * per, generator=gen(9)).int().view(3, per)
    table[2, 0] = -1                                   # a page that is not there
    start, count = [0, page - 1 if page < 40 else 40, 0], [T, 5, T]
    k, v = randn(1, B, T, heads, dim, dtype=dtype), randn(2, B, T, heads, dim, dtype=dtype)
    k[0, 3], v[0, 4] = 0.0, 0.0
    k[0, 5, 0, 7] = math.inf
    v[0, 6, 0, 2] = math.nan
    rot = dim // 2
    phase, _ = lm.rope_phases(rot)
    pos = torch.randint(0, 5000, (B, T), generator=gen(3)).int().cuda()
    lm.fa_cache_write(cache, k, v, table.cuda(), i32(start), i32(count), pos, phase, interleaved=page == 16)
    turned = np.stack([ref.rope(k[b], pos[b], rot, interleaved=page == 16) for b in range(B)])
    out = [torch.full((B, 64, heads, dim), 7.0, device="cuda") for _ in range(2)]
    lm.fa_cache_read(cache, table.cuda(), i32([start[b] + count[b] for b in range(B)]), *out)
    written = torch.zeros(cache.k.shape[:3], dtype=torch.bool)
    for b in range(B):
        for j in range(count[b]):
            slot = start[b] + j
            p = int(table[b, slot // page])
            if p < 0:
                assert (out[0][b, slot] == 0).all() and (out[1][b, slot] == 0).all()
                continue
            written[p, :, slot % page] = True
            for name, want, got in (("k", turned[b, j], out[0][b, slot]), ("v", v[b, j].double().cpu().numpy(), out[1][b, slot])):
                got = got.double().cpu().numpy()
                size = ref.pair_sum(k[b, j][None], rot, page == 16)[0] if name == "k" else 0.0
                if fmt != F8:
                    fine = np.isfinite(want)
                    tol = 1.5e-6 * np.where(np.isfinite(size), size, 0) + ref.HALF_ULP[fmt] * np.abs(want) + ref.TINY[fmt]
                    if fmt == HF:
                        fine &= np.abs(want) < 65000
                    assert (np.abs(got[fine] - want[fine]) <= tol[fine]).all()
                    continue
                for h in range(heads):
                    w, g = want[h], got[h]
                    if not np.isfinite(w).all():
                        assert np.isnan(g).all()                    # the row is marked
                        continue
                    scale = float((cache.k_scale if name == "k" else cache.v_scale)[p, h, slot % page])
                    assert abs(scale - np.abs(w).max() / 448) <= 2e-6 * np.abs(w).max() / 448
                    # half a step of an 8-bit value: 2^-4 of it, or 2^-10 below 2^-6; the scale's own
                    # rounding and the read's shift both by a few 2^-24
                    tol = scale * np.maximum(np.abs(w) / max(scale, 1e-30) * 2.0 ** -4, 2.0 ** -10) * (1 + 1e-5) + 2e-6 * np.abs(w).max()
                    assert (np.abs(g - w) <= tol).all()
    assert (out[0][0, T:] == 0).all() and (out[1][1, start[1] + 5:] == 0).all()
    for x, old in zip(cache, before):                  # the other slots were left alone
        if x is not None:
            assert torch.equal(x.view(torch.uint8).view(*x.shape[:3], -1).cpu()[~written],
                               old.view(torch.uint8).view(*x.shape[:3], -1).cpu()[~written])


@pytest.mark.parametrize("dtype", [HF, BF])
def test_cache_write_strided(dtype):
    """The keys and values of a fused projection, not 16-byte aligned either."""
    wide = randn(4, 2, 9, 7, 70, dtype=dtype)
    k, v = wide[:, :, 1:4, 3:67], wide[:, :, 4:7, 5:69]
    got = []
    table = i32([[2, 0], [1, 3]])
    for a, b in ((k, v), (k.contiguous(), v.contiguous())):
        cache = lm.KVCache.empty(4, 3, 8, 64, F8)
        for x in cache:
            x.view(torch.uint8).zero_()
        lm.fa_cache_write(cache, a, b, table, i32([3, 0]))
        got.append(cache)
    for x, y in zip(*got):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


def test_cache_read_types():
    for fmt in (HF, BF, F8):
        cache, table = make_cache(3, 2, 70, 2, 16, 48, fmt)
        outs = [[torch.empty((2, 70, 2, 48), dtype=d, device="cuda") for _ in range(2)] for d in (FP, HF, BF)]
        for o in outs:
            lm.fa_cache_read(cache, table, i32([70, 33]), *o)
        for b, n in ((0, 70), (1, 33)):
            for x, want in zip(outs[0], ref.cached_rows(cache, table.cpu(), b, n)):
                np.testing.assert_allclose(x[b, :n].double().cpu(), want, rtol=2.0 ** -23)
        for o in outs[1:]:
            for x, y in zip(o, outs[0]):
                assert torch.equal(x, y.to(x.dtype))


@pytest.mark.parametrize("fmt", [BF, F8])
@pytest.mark.parametrize("page", [4, 16])
def test_cache_keep(fmt, page):
    cache, table = make_cache(5, 3, 40, 2, page, 64, fmt)
    old = [None if x is None else x.clone() for x in cache]
    length = [7, 0, 15]
    path = [[0, 2, 5, 6, 11, -1, 3], [1, 4, 3, 9, -1, -1, -1], [-1, 1, 2, 3, 4, 5, 6]]
    kept = [[0, 2, 5, 6, 11], [1, 4], []]              # 3 does not ascend: the path ends
    lm.fa_cache_keep(cache, table, i32(length), i32(path))
    t = table.cpu()
    for x, was in zip(cache, old):
        if x is None:
            continue
        bits = {1: torch.uint8, 2: torch.int16, 4: torch.int32}[x.element_size()]
        was = was.view(bits)
        want = was.clone()
        for b in range(3):
            for i, j in enumerate(kept[b]):
                to, fr = length[b] + i, length[b] + j
                want[int(t[b, to // page]), :, to % page] = was[int(t[b, fr // page]), :, fr % page]
        assert torch.equal(x.view(bits), want)


# ------------------------------------------------------------------ trees and attention

@pytest.mark.parametrize("T", [1, 2, 63, 64, 65, 200, 1024])
def test_tree_mask(T):
    rng = np.random.default_rng(T)
    parents = np.stack([np.arange(T) - 1, np.full(T, -1), [rng.integers(-1, max(j, 1)) if j else -1 for j in range(T)]])
    parents[1, T // 2:] = T + 5                        # not an earlier token: a root
    mask, depth = lm.fa_tree_mask(i32(parents))
    m, d = mask.cpu().numpy().astype(np.uint64), depth.cpu().numpy()
    for b in range(3):
        for j, seen in enumerate(ref.tree_seen(parents[b].tolist())):
            bits = {64 * w + i for w in range(m.shape[2]) for i in range(64) if int(m[b, j, w]) >> i & 1}
            assert bits == seen and d[b, j] == len(seen) - 1


def words(seen, T):
    """Mask words from a boolean [B, T, T] array."""
    B = seen.shape[0]
    out = np.zeros((B, T, (T + 63) // 64), np.uint64)
    for b, i, j in zip(*np.nonzero(seen)):
        out[b, i, j // 64] |= np.uint64(1) << np.uint64(j % 64)
    return torch.from_numpy(out.astype(np.int64)).cuda()


def check_attention(q, cache, table, length, mask=None, count=None, scale=None, attend=None):
    B, T, H, D = q.shape
    attend = attend or lm.TreeAttention(B, T, H, cache.k.shape[1], D, q.dtype)
    attend.out.fill_(9.0)
    attend.lse.fill_(9.0)
    out, lse = attend(q, cache, table, i32(length), mask, None if count is None else i32(count), scale)
    got, gl = out.double().cpu().numpy(), lse.double().cpu().numpy()
    want, wl, weight, size = ref.attention(q, cache, table, length, None if mask is None else mask.cpu(), count, scale)
    ds = 2.0 ** -17 * size
    u = 2.0 ** -8 if cache.k.dtype == BF else 2.0 ** -10
    tol = (u + 4 * ds[..., None]) * weight + ref.HALF_ULP[q.dtype] * np.abs(want) + ref.TINY[q.dtype]
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (np.argwhere(bad)[:3], got[bad][:3], want[bad][:3], tol[bad][:3])
    empty = np.isneginf(wl)
    assert np.array_equal(empty, np.isneginf(gl))
    seen = ~empty
    assert (np.abs(gl[seen] - wl[seen]) <= ds[seen] + 4e-6 * np.maximum(1, np.abs(wl[seen]))).all()
    assert (got[empty] == 0).all()
    return out, lse


LENGTHS = [0, 1, 15, 64, 127, 128, 129, 300]


@pytest.mark.parametrize("fmt,dtype", [(BF, BF), (HF, HF), (F8, BF), (F8, HF)])
@pytest.mark.parametrize("T,heads,kv,dim,page", [(1, 4, 1, 64, 16), (1, 8, 8, 128, 64), (3, 6, 2, 128, 1), (17, 8, 4, 96, 32),
                                                 (64, 4, 2, 128, 128), (5, 7, 1, 16, 8), (70, 5, 1, 80, 16)])
def test_attention(fmt, dtype, T, heads, kv, dim, page):
    B = len(LENGTHS)
    cache, table = make_cache(T + dim, B, max(LENGTHS) + T, kv, page, dim, fmt)
    rng = np.random.default_rng(T)
    q = randn(T, B, T, heads, dim, dtype=dtype, scale=1.5)
    parents = np.stack([[int(rng.integers(-1, j)) if j else -1 for j in range(T)] for _ in range(B)])
    mask, _ = lm.fa_tree_mask(i32(parents))
    count = [max(0, T - b % 4) for b in range(B)]
    check_attention(q, cache, table, LENGTHS, mask, count)
    check_attention(q, cache, table, LENGTHS)
    seen = rng.random((B, T, T)) < 0.3                 # rows that see nothing of the draft, or nothing at all
    seen[:, 0] = False
    check_attention(q, cache, table, LENGTHS, words(seen, T), None, 0.3)


@pytest.mark.parametrize("fmt,dtype", [(BF, BF), (F8, HF)])
@pytest.mark.parametrize("T,heads,kv", [(1, 8, 2), (16, 4, 1), (40, 8, 1), (130, 3, 1), (200, 2, 1)])
def test_attention_rows_and_long_lengths(fmt, dtype, T, heads, kv):
    """Row counts across the kernel's tiles, contexts long enough to be split."""
    length = [2500, 1029]
    cache, table = make_cache(T, 2, 2500 + T, kv, 64, 128, fmt)
    q = randn(T + 1, 2, T, heads, 128, dtype=dtype, scale=1.5)
    parents = np.tile(np.arange(T) - 1, (2, 1))
    mask, _ = lm.fa_tree_mask(i32(parents))
    a = check_attention(q, cache, table, length, mask)
    a = [x.clone() for x in a]
    b = check_attention(q, cache, table, length, mask)
    assert all(torch.equal(x, y) for x, y in zip(a, b))   # the same call gives the same bits


def test_attention_large_and_peaked_values():
    """Scores of hundreds, growing and shrinking along the context; values and scales of very
    different sizes."""
    for fmt, dtype in ((BF, BF), (HF, HF), (F8, BF), (F8, HF)):
        cache, table = make_cache(8, 2, 1200, 2, 16, 64, fmt)
        ramp = torch.ones(1200)
        ramp[:600] = torch.linspace(0.01, 12.0, 600)
        ramp[600:] = torch.linspace(12.0, 0.01, 600)
        for b in range(2):
            for t in range(1200):
                p, g = int(table[b, t // 16]), t % 16
                if fmt == F8:
                    cache.k_scale[p, :, g] *= float(ramp[t])
                    cache.v_scale[p, :, g] *= float(ramp[1199 - t]) * (1e4 if t > 900 else 1e-3)
                else:
                    cache.k[p, :, g] *= float(ramp[t])
                    cache.v[p, :, g] *= float(ramp[1199 - t]) * (100.0 if t > 900 else 1e-2)
        q = randn(11, 2, 3, 4, 64, dtype=dtype, scale=8.0)
        check_attention(q, cache, table, [1190, 700], None, None)


@pytest.mark.parametrize("fmt,dtype", [(BF, BF), (HF, HF), (F8, BF)])
def test_attention_ignores_what_is_not_seen(fmt, dtype):
    """NaN and infinities in slots past the end, in unused pages, in unused drafted tokens and in
    drafted tokens that a row does not see change nothing; a row that sees one is not finite."""
    T, n = 6, [0, 130]
    cache, table = make_cache(4, 2, 140, 1, 16, 64, fmt)
    q = randn(2, 2, T, 3, 64, dtype=dtype)
    seen = np.tile(np.tril(np.ones((T, T), bool)), (2, 1, 1))
    seen[:, :, 2] = False
    seen[:, 2, 2] = True                               # only token 2 sees token 2
    mask = words(seen, T)
    clean, lse = check_attention(q, cache, table, n, mask, [5, 5])
    clean, lse = clean.clone(), lse.clone()
    for bad in (math.nan, math.inf, -math.inf):
        for b in range(2):
            for slot in [n[b] + 2] + list(range(n[b] + 5, table.shape[1] * 16)):
                p, g = int(table[b, slot // 16]), slot % 16
                if fmt == F8:
                    cache.k_scale[p, :, g] = cache.v_scale[p, :, g] = bad
                else:
                    cache.k[p, :, g, 3] = cache.v[p, :, g, 5] = bad
        out, l2 = lm.TreeAttention(2, T, 3, 1, 64, dtype)(q, cache, table, i32(n), mask, i32([5, 5]))
        keep = [0, 1, 3, 4, 5]
        assert torch.equal(out[:, keep], clean[:, keep]) and torch.equal(l2[:, keep], lse[:, keep])
        if math.isnan(bad):
            assert not torch.isfinite(out[:, 2]).all(dim=-1).any()


def test_attention_missing_pages_and_short_tables():
    cache, table = make_cache(6, 2, 100, 2, 16, 64, BF)
    table[0, 1], table[1, 0], table[1, 3] = -1, cache.k.shape[0], 2 ** 30
    q = randn(3, 2, 2, 4, 64, dtype=BF)
    check_attention(q, cache, table, [98, 60])
    check_attention(q, cache, table, [500, 400])       # lengths past the table's end


def test_attention_strided_queries_and_streams():
    cache, table = make_cache(7, 2, 50, 2, 16, 64, F8)
    wide = randn(5, 2, 3, 9, 72, dtype=BF)
    q = wide[:, :, 1:5, 8:]
    want, _ = check_attention(q.contiguous(), cache, table, [40, 17])
    want = want.clone()
    side = torch.cuda.Stream()
    attend = lm.TreeAttention(2, 3, 4, 2, 64, BF)
    length = i32([40, 17])
    side.wait_stream(torch.cuda.current_stream())
    out, _ = attend(q, cache, table, length, stream=side)
    side.synchronize()
    assert torch.equal(out, want)
    with torch.cuda.stream(side):
        out, _ = attend(q, cache, table, length)
    side.synchronize()
    assert torch.equal(out, want)


def test_operators_in_a_graph():
    """A decoding step's calls can be captured and replayed with new data in place."""
    cache, table = make_cache(9, 2, 200, 2, 16, 64, F8)
    attend, length = lm.TreeAttention(2, 1, 4, 2, 64, BF), i32([100, 3])
    q, k, v = randn(1, 2, 1, 4, 64, dtype=BF), randn(2, 2, 1, 2, 64, dtype=BF), randn(3, 2, 1, 2, 64, dtype=BF)
    phase, _ = lm.rope_phases(64)
    pos = length[:, None].contiguous()
    turned = torch.empty_like(q)

    def step():
        lm.fa_rope(q.view(2, 4, 64), pos.view(2), phase, out=turned.view(2, 4, 64))
        lm.fa_cache_write(cache, k, v, table, length, None, pos, phase)
        attend(turned, cache, table, length)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    length += 1
    pos += 1
    q.copy_(randn(5, 2, 1, 4, 64, dtype=BF))
    graph.replay()
    torch.cuda.synchronize()
    got = attend.out.clone()
    step()
    assert torch.equal(got, attend.out)


# ------------------------------------------------------------------ beams

def check_beam(logp, scores, top, states=None, nxt=None, live=None):
    N, K, V = logp.shape
    got = lm.BeamSelect(N, K, V, top, logp.dtype)(logp, scores, states, nxt, live)
    want = ref.beam(logp, scores, top, None if states is None else states.cpu().numpy(), None if nxt is None else nxt.cpu().numpy())
    for g, w in zip(got, want):
        if g is not None:
            assert np.array_equal(g.cpu().numpy(), w)
    return got


@pytest.mark.parametrize("dtype", [FP, HF, BF])
@pytest.mark.parametrize("N,K,V,top", [(1, 1, 1, 1), (2, 3, 7, 30), (1, 4, 32000, 4), (3, 2, 8191, 256), (2, 5, 8193, 10),
                                       (1, 16, 20001, 33), (2, 1, 100, 100)])
def test_beam_select(dtype, N, K, V, top):
    logp = torch.log_softmax(3 * torch.randn((N, K, V), generator=gen(V)), -1).to(dtype).cuda()
    scores = -5 * torch.rand((N, K), generator=gen(1)).cuda()
    check_beam(logp, scores, top)
    coarse = (logp.float() * 2).round() / 2            # many ties, and -0
    check_beam(coarse.to(dtype), (scores * 2).round() / 2, top)


def test_beam_select_adversarial_order():
    """Ascending values (every cell beats the ones before it), all equal, all but a few dead."""
    for top in (1, 16, 256):
        up = torch.arange(3 * 30000, dtype=FP).view(1, 3, 30000).cuda()
        check_beam(up, torch.zeros((1, 3)).cuda(), top)
        check_beam(torch.zeros((2, 3, 30000), device="cuda"), torch.zeros((2, 3)).cuda(), top)
        one = torch.full((2, 3, 30000), -math.inf, device="cuda")
        one[:, 1, 29999], one[1, 0, 5], one[1, 2, 7] = 1.0, math.nan, math.inf
        check_beam(one, torch.zeros((2, 3)).cuda(), top)
        scores = torch.tensor([[-math.inf, 0.0, math.nan]]).cuda()
        check_beam(up, scores, top)


@pytest.mark.parametrize("dtype", [FP, BF])
@pytest.mark.parametrize("offset", [0, 1, 5])
def test_beam_select_strided_rows(dtype, offset):
    wide = torch.randn((2, 6, 9001), generator=gen(2)).to(dtype).cuda()
    logp = wide[:, ::2, offset:offset + 8500]
    check_beam(logp, torch.zeros((2, 3)).cuda(), 12)


@pytest.mark.parametrize("make", [synth.real_number_dfa, lambda: synth.random_dfa(64, 3001, 0.7, 8, 1),
                                  lambda: synth.layered_chain(40, 9000, 3), lambda: synth.single_state_fa(50)])
def test_beam_select_under_an_automaton(make):
    fa = make()
    aut = native.fa_compile(fa)
    nxt, live = lm.fa_beam_tables(aut)
    S, V = fa.n_states, fa.vocab
    table = np.full((S, V), -1, np.int64)
    for e in range(fa.n_edges):
        table[fa.edge_src[e], fa.labels(e)] = fa.edge_dst[e]
    reach = np.zeros(S, bool)
    reach[fa.accept] = True
    for _ in range(S):
        for e in range(fa.n_edges):
            reach[fa.edge_src[e]] |= reach[fa.edge_dst[e]]
    table[(table >= 0) & ~reach[table]] = -1
    assert np.array_equal(nxt.cpu().numpy(), table)
    bits = live.cpu().numpy().view(np.uint32)
    for s in range(S):
        got = [(int(bits[s, v // 32]) >> (v % 32)) & 1 for v in range(V)]
        assert np.array_equal(np.array(got, bool), table[s] >= 0)
        assert V % 32 == 0 or int(bits[s, -1]) >> (V % 32) == 0
    rng = np.random.default_rng(0)
    states = i32(rng.integers(0, S, (2, 4)))
    states[0, 1], states[1, 2] = -1, S                 # dead beams
    logp = torch.randn((2, 4, V), generator=gen(3)).cuda()
    check_beam(logp, -torch.rand((2, 4), generator=gen(4)).cuda(), 6, states, nxt, live)


def test_beam_tables_without_an_accepting_state_and_for_an_nfa():
    fa = synth.random_dfa(5, 40, 0.5, 1, 3)
    fa.accept = np.zeros(0, np.int32)
    nxt, live = lm.fa_beam_tables(native.fa_compile(fa))
    assert (nxt == -1).all() and (live == 0).all()
    with pytest.raises(native.FaError) as e:
        lm.fa_beam_tables(native.fa_compile(synth.real_number_dfa().duplicated_edges()))
    assert e.value.code == native.FA_ERR_UNSUPPORTED


@pytest.mark.parametrize("W", [1, 3, 128, 5000])
def test_beam_reorder(W):
    src = torch.randint(0, 1000, (2, 3, W), generator=gen(W)).int().cuda()
    parent, token = i32([[2, 0, 0, -1], [1, 3, 2, 1]]), i32([[5, 6, 7, -1], [8, -1, 9, 10]])
    for at in (0, W - 1):
        for tok in (token, None):
            got = lm.fa_beam_reorder(src, parent, token=tok, at=at).cpu().numpy()
            for n in range(2):
                for k in range(4):
                    p = int(parent[n, k])
                    want = src[n, p].cpu().numpy().copy() if 0 <= p < 3 else np.full(W, -1, np.int32)
                    if tok is not None:
                        want[at] = int(token[n, k])
                    assert np.array_equal(got[n, k], want)


# ------------------------------------------------------------------ refusals

def test_refusals_on_tensors():
    x, pos = randn(0, 4, 2, 16), i32([0, 1, 2, 3])
    phase, _ = lm.rope_phases(16)
    with pytest.raises(TypeError):
        lm.fa_rope(x.double(), pos, phase)
    with pytest.raises(TypeError):
        lm.fa_rope(x.cpu(), pos, phase)
    with pytest.raises(ValueError):
        lm.fa_rope(x, pos[:3], phase)
    with pytest.raises(ValueError):
        lm.fa_rope(x.transpose(1, 2), pos, lm.rope_phases(2)[0])
    with pytest.raises(native.FaError):
        lm.fa_rope(x, pos, lm.rope_phases(18)[0])
    cache, table = make_cache(1, 2, 30, 2, 16, 64, BF)
    q = randn(1, 2, 1, 4, 64, dtype=HF)
    with pytest.raises(native.FaError) as e:
        lm.TreeAttention(2, 1, 4, 2, 64, HF)(q, cache, table, i32([1, 1]))
    assert e.value.code == native.FA_ERR_UNSUPPORTED
    with pytest.raises(TypeError):
        lm.TreeAttention(2, 1, 4, 2, 64, BF)(q, cache, table, i32([1, 1]))
    with pytest.raises(ValueError):
        lm.TreeAttention(2, 1, 4, 2, 64, HF)(q, cache, table, i32([1, 1, 1]))
    wide = torch.zeros((2, 1, 4, 68), dtype=BF, device="cuda")[..., 4:]
    with pytest.raises(native.FaError):
        lm.TreeAttention(2, 1, 4, 2, 64, BF)(wide, cache, table, i32([1, 1]))
    with pytest.raises(ValueError):
        lm.KVCache(cache.k, cache.v, cache.k[..., 0].float(), None).describe()
    with pytest.raises(ValueError):
        lm.fa_cache_write(cache, randn(0, 2, 1, 3, 64), randn(0, 2, 1, 3, 64), table, i32([0, 0]))
    with pytest.raises(native.FaError) as e:
        short = lm.BeamSelect(1, 64, 30000, 8)
        short.workspace = short.workspace[:256]
        short(torch.zeros((1, 64, 30000), device="cuda"), torch.zeros((1, 64), device="cuda"))
    assert e.value.code == native.FA_ERR_WORKSPACE_TOO_SMALL
