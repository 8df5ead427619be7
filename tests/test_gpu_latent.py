"""The latent cache's writes and moves and the attention over it, against plain 64-bit implementations.

Tolerances, from the roundings: a written element is rounded once (half a unit of its type), a rotated one also carries the
fp32 error of its angle (2^-26 turn) and of three operations, 2^-21 of |x0| + |x1| in all.  With
ds = 2^-17 max_t scale sum_d |q_d c_d| for the error of a score (fp32 sums of up to 576 products, and the exponential's
argument and value) and w = sum_t p |c'|, a result is off by at most (u + 4 ds) w, u = 2^-8 for weights in bf16
and 2^-10 in fp16, plus its own rounding."""
import pytest

torch = pytest.importorskip("torch")

import serving_reference as ref  # noqa: E402
from constrained_decoding_diffusion_gb300 import lm  # noqa: E402

pytestmark = pytest.mark.gpu

F32, BF, HF = torch.float32, torch.bfloat16, torch.float16


def ints(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


def normal(seed, *shape, dtype=F32):
    return torch.randn(shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").to(dtype)


# ------------------------------------------------------------------ writes

@pytest.mark.parametrize("src", [F32, BF, HF])
@pytest.mark.parametrize("dst", [BF, HF])
@pytest.mark.parametrize("latent,rope,inter", [(128, 16, False), (256, 32, True), (384, 48, False), (512, 64, True), (512, 64, False)])
def test_write(src, dst, latent, rope, inter):
    for N, wide in ((1, 0), (5, 8), (67, 3), (300, 0)):
        cache = lm.LatentCache(normal(1, 41, 8, latent + rope, dtype=dst), latent)
        before = cache.rows.clone()
        down = normal(2, N, latent + rope + wide, dtype=src)
        x, key = down[:, :latent], down[:, latent:latent + rope]
        slot = torch.randperm(41 * 8, generator=torch.Generator().manual_seed(N))[:N].int().cuda()
        slot[N // 2] = -1
        if N > 5:
            slot[3], slot[4], slot[5] = 41 * 8, 2 ** 31 - 1, -2 ** 31
        pos = torch.randint(-5, 2 ** 31 - 1, (N,), generator=torch.Generator().manual_seed(N)).int().cuda()
        phase, _ = lm.rope_phases(rope)
        lm.fa_latent_write(cache, x, key, slot, pos % 100000, phase, inter, 1.25)
        ok = ((slot >= 0) & (slot < 41 * 8)).cpu()
        want = before.clone().double().view(-1, latent + rope).cpu()
        size = torch.zeros_like(want)
        turned = torch.from_numpy(ref.rotated(key, pos % 100000, interleaved=inter, mscale=1.25))
        at = slot.cpu().long()[ok]
        want[at] = torch.cat([x.double().cpu(), turned], 1)[ok]
        size[at, latent:] = key.double().abs().cpu().max(1, keepdim=True).values[ok]
        err = (cache.rows.double().cpu().view_as(want) - want).abs()
        rounding = ref.HALF_ULP[dst] * want.abs() + ref.TINY[dst]
        untouched = torch.ones(41 * 8, dtype=torch.bool)
        untouched[at] = False
        assert (err[untouched] == 0).all()
        assert (err <= rounding + 1.25 * 2.0 ** -20 * size).all()


def test_write_without_positions():
    cache = lm.LatentCache.empty(4, 16, 128, 32, HF)
    x, key = normal(1, 9, 128, dtype=HF), normal(2, 9, 32, dtype=HF)
    slot = ints([63, 0, 5, 17, 33, 2, 1, 8, 62])
    lm.fa_latent_write(cache, x, key, slot)
    assert torch.equal(cache.rows.view(64, 160)[slot.long()], torch.cat([x, key], 1))


def test_write_refuses_phases_of_another_size():
    cache = lm.LatentCache.empty(4, 16, 128, 32, HF)
    x, key = normal(1, 3, 128, dtype=HF), normal(2, 3, 32, dtype=HF)
    with pytest.raises(ValueError):
        lm.fa_latent_write(cache, x, key, ints([0, 1, 2]), ints([0, 1, 2]), lm.rope_phases(64)[0])
    with pytest.raises(ValueError):
        lm.fa_latent_write(cache, x, key[:, :16], ints([0, 1, 2]))
    with pytest.raises(TypeError):
        lm.fa_latent_write(cache, x, key.float(), ints([0, 1, 2]))
    with pytest.raises(TypeError):
        lm.LatentCache.empty(4, 16, 128, 32, torch.float8_e4m3fn)


@pytest.mark.parametrize("size", [1, 4, 64])
def test_keep(size):
    """Paths of any length, ended anywhere; entries that do not ascend end a path; slots without a page read as zeros
    and take nothing."""
    P, B = 21, 7
    per = -(-60 // size)
    cache = lm.LatentCache(normal(3, B * per + 2, size, 144, dtype=BF), 128)
    table = torch.randperm(B * per + 2, generator=torch.Generator().manual_seed(size))[:B * per].int().view(B, per)
    table[5, 25 // size] = -1
    table[6, 30 // size] = B * per + 2
    length = [0, 7, 39, 12, 33, 20, 17]
    paths = [[0, 2, 3, 7, 20], [], list(range(P)), [1, 2, 5, 5, 6], [3, 4, 2, 9], list(range(1, P)), [0, 4, 9, 11, 13, 14, 17]]
    path = torch.full((B, P), -1, dtype=torch.int32)
    for b, p in enumerate(paths):
        path[b, :len(p)] = torch.tensor(p, dtype=torch.int32)
    want = cache.rows.clone().cpu()
    for b, p in enumerate(paths):
        def place(t):
            page = int(table[b, t // size]) if t // size < per else -1
            return (page, t % size) if 0 <= page < want.shape[0] else None
        last = -1
        for i, j in enumerate(p):
            if j <= last:
                break
            last = j
            src, dst = place(length[b] + j), place(length[b] + i)
            if dst is not None and i != j:
                want[dst] = want[src].clone() if src is not None else 0
    lm.fa_latent_keep(cache, table.cuda(), ints(length), path.cuda())
    assert torch.equal(cache.rows.cpu(), want)


# ------------------------------------------------------------------ attention

def make(seed, length, T, size, latent, rope, dtype, spare=3):
    B, per = len(length), max(1, -(-(max(length) + T) // size))
    n = B * per + spare
    table = torch.randperm(n, generator=torch.Generator().manual_seed(seed))[:B * per].int().view(B, per).cuda()
    return lm.LatentCache(normal(seed, n, size, latent + rope, dtype=dtype), latent), table


def chains(B, T):
    return lm.fa_tree_mask(torch.arange(-1, T - 1, dtype=torch.int32).expand(B, T).contiguous().cuda())[0]


def trees(seed, B, T):
    g = torch.Generator().manual_seed(seed)
    return lm.fa_tree_mask(((torch.rand(B, T, generator=g) * (torch.arange(T) + 1)).int() - 1).cuda())[0]


def check(q, cache, table, length, scale, mask=None, count=None, attend=None):
    B, T, H, D = q.shape
    length, count = ints(length), None if count is None else ints(count)
    attend = attend or lm.LatentAttention(B, T, H, cache.latent_dim, D - cache.latent_dim, q.dtype)
    attend.out.fill_(9.0)
    attend.lse.fill_(9.0)
    out, lse = attend(q, cache, table, length, scale, mask, count)
    want, wl, w, size = ref.latent_attention(q, cache.rows, cache.latent_dim, table, length, scale, mask, count)
    ds = 2.0 ** -17 * size
    u = 2.0 ** -8 if q.dtype == BF else 2.0 ** -10
    tol = (u + 4 * ds[..., None]) * w + ref.HALF_ULP[q.dtype] * want.abs() + ref.TINY[q.dtype]
    assert ((out.double() - want).abs() <= tol).all()
    assert torch.equal(torch.isneginf(lse), torch.isneginf(wl))
    some = ~torch.isneginf(wl)
    assert ((lse.double() - wl).abs()[some] <= (ds + 4e-6 * wl.abs().clamp_min(1))[some]).all()
    assert (out[~some] == 0).all()
    return out.clone(), lse.clone()


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("latent,rope", [(128, 16), (256, 32), (384, 48), (512, 64)])
@pytest.mark.parametrize("T,H,size", [(1, 1, 16), (1, 16, 64), (3, 5, 8), (2, 40, 32), (1, 128, 128), (9, 16, 4)])
def test_ragged_lengths(dtype, latent, rope, T, H, size):
    length = [0, 1, 63, 64, 65, 300, 511, 129 - T]
    cache, table = make(latent + T, length, T, size, latent, rope, dtype)
    q = normal(H, len(length), T, H, latent + rope, dtype=dtype)
    args = (q, cache, table, length, 0.07, chains(len(length), T))
    first = check(*args)
    assert all(torch.equal(x, y) for x, y in zip(first, check(*args)))


@pytest.mark.parametrize("T", [1, 2, 16, 63, 64, 65, 130])
@pytest.mark.parametrize("how", ["tree", "block"])
def test_drafts(T, how):
    length = [0, 70, 190, 3]
    cache, table = make(T, length, T, 16, 128, 32, BF)
    q = normal(T, 4, T, 3, 160, dtype=BF)
    mask = trees(T, 4, T) if how == "tree" else None
    check(q, cache, table, length, 0.1, mask)
    check(q, cache, table, length, 0.1, mask, count=[0, T, (T + 1) // 2, 1])
    check(q, cache, table, length, 0.1, mask, count=[-4, T + 9, 1, T])


def test_masks_that_leave_rows_empty():
    length = [0, 0, 40]
    cache, table = make(2, length, 6, 8, 256, 64, HF)
    mask = torch.zeros(3, 6, 1, dtype=torch.int64, device="cuda")
    mask[1, :, 0] = torch.tensor([0, 1, 2, 0, 63, -1])
    out, lse = check(normal(3, 3, 6, 4, 320, dtype=HF), cache, table, length, 0.06, mask)
    assert torch.isneginf(lse[0]).all() and torch.isneginf(lse[1, 0]).all() and torch.isfinite(lse[2]).all()


@pytest.mark.parametrize("T,H", [(1, 16), (8, 16)])
def test_pages_that_are_none(T, H):
    """Slots without a page are not attended to, at the start, in the middle, at the end and everywhere."""
    length = [200, 200, 200, 150, 90]
    cache, table = make(5, length, T, 16, 512, 64, BF)
    table[0, 0] = -1
    table[1, 5:8] = cache.rows.shape[0]
    table[2, 12:] = -1
    table[3] = -1
    table[4, ::2] = -2 ** 31
    _, lse = check(normal(1, 5, T, H, 576, dtype=BF), cache, table, length, 0.05, chains(5, T))
    assert torch.isneginf(lse[3]).all()


def test_lengths_past_the_table():
    cache, table = make(6, [64, 64, 64], 4, 16, 128, 16, HF, spare=0)
    table = table[:, :4].contiguous()
    check(normal(2, 3, 4, 6, 144, dtype=HF), cache, table, [64, 62, 1000], 0.1, chains(3, 4))
    q = normal(2, 3, 4, 6, 144, dtype=HF)
    out, lse = lm.LatentAttention(3, 4, 6, 128, 16, HF)(q, cache, table[:, :0], ints([5, 0, 9]), 0.1)
    assert (out == 0).all() and torch.isneginf(lse).all()


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("T", [4, 70])
def test_hidden_values_have_no_part(bad, T):
    """Drafted slots that a row does not see, slots past the draft and pages of no sequence may hold anything."""
    length = [100, 0, 250]
    cache, table = make(7, length, T, 32, 256, 32, BF)
    mask = chains(3, T)
    q = normal(4, 3, T, 5, 288, dtype=BF)
    args = (q, cache, table, length, 0.06, mask, [T, T - 1, T])
    want = check(*args)
    used = torch.zeros(cache.rows.shape[:2], dtype=torch.bool, device="cuda")
    for b, n in enumerate(length):
        for t in range(n + (T - 1 if b == 1 else T)):
            used[table[b, t // 32], t % 32] = True
    cache.rows[~used] = bad
    assert all(torch.equal(x, y) for x, y in zip(want, check(*args)))
    # the third drafted slot: only the rows from the third on see it
    for b, n in enumerate(length):
        cache.rows[table[b, (n + 2) // 32], (n + 2) % 32, 17 if b else 270] = bad
    attend = lm.LatentAttention(3, T, 5, 256, 32, BF)
    out, lse = attend(q, cache, table, ints(length), 0.06, mask, ints([T, T - 1, T]))
    assert torch.equal(out[:, :2], want[0][:, :2]) and torch.equal(lse[:, :2], want[1][:, :2])


@pytest.mark.parametrize("T,H", [(1, 8), (20, 8)])
@pytest.mark.parametrize("size", [2.0 ** -10, 30.0, 1000.0])
def test_scores_of_any_size(T, H, size):
    """Largest scores that come first, last or in the middle of the slots."""
    length = [700, 300, 65]
    cache, table = make(8, length, T, 16, 256, 64, BF)
    q = normal(5, 3, T, H, 320, dtype=BF)
    for b, t in ((0, 699), (1, 0), (2, 30)):
        cache.rows[table[b, t // 16], t % 16] = q[b, 0, 0]
    check((q * size).to(BF), cache, table, length, 0.06, chains(3, T))


def test_scores_that_rise_slot_by_slot():
    """Every tile moves the running maximum, for some rows up and for some down."""
    n = 640
    cache, table = make(9, [n], 1, 64, 128, 16, HF)
    cache.rows.mul_(0.05)
    ramp = torch.arange(n, device="cuda") / 16.0
    cache.rows.view(-1, 144)[(table[0].long() * 64).repeat_interleave(64)[:n] + torch.arange(n, device="cuda") % 64, 0] = ramp.to(HF)
    q = normal(6, 1, 1, 64, 144, dtype=HF)
    q[0, 0, :, 0] = torch.linspace(-8, 8, 64, device="cuda").to(HF)
    check(q, cache, table, [n], 1.0)


def test_zero_queries_weigh_all_alike():
    length = [300, 1]
    cache, table = make(10, length, 1, 32, 512, 64, BF)
    _, lse = check(torch.zeros(2, 1, 16, 576, dtype=BF, device="cuda"), cache, table, length, 0.07)
    seen = torch.tensor([301.0, 2.0], device="cuda").log().view(2, 1, 1)
    assert (lse - seen).abs().max() <= 4e-6 * 8


@pytest.mark.parametrize("H", [1, 16])
def test_strides(H):
    """Queries that are parts of wider buffers, in any order."""
    length = [90, 33]
    cache, table = make(11, length, 3, 16, 256, 32, BF)
    q = normal(7, 2, 3, H, 288, dtype=BF)
    want = check(q, cache, table, length, 0.07)
    wide = torch.full((3, 2, H, 288 + 24), float("nan"), dtype=BF, device="cuda")
    wide[..., 8:296] = q.transpose(0, 1)
    assert all(torch.equal(x, y) for x, y in zip(want, check(wide[..., 8:296].transpose(0, 1), cache, table, length, 0.07)))
    same = q[:, :1].expand(2, 3, H, 288)
    check(same, cache, table, length, 0.07)
    with pytest.raises(Exception):
        lm.LatentAttention(2, 3, H, 256, 32, BF)(wide[..., 4:292].transpose(0, 1), cache, table, ints(length), 0.07)


def test_one_token_of_one_head_whose_strides_mean_nothing():
    cache, table = make(12, [50], 1, 16, 128, 16, HF)
    q = normal(8, 1, 1, 1, 144, dtype=HF).as_strided((1, 1, 1, 144), (1, 3, 5, 1))
    check(q, cache, table, [50], 0.1)


@pytest.mark.parametrize("T,H", [(1, 16), (1, 70), (4, 16)])
def test_hundreds_of_short_sequences(T, H):
    B = 333
    length = [(7 * b * b) % 150 if b % 5 else 0 for b in range(B)]
    cache, table = make(13, length, T, 16, 128, 16, BF)
    check(normal(9, B, T, H, 144, dtype=BF), cache, table, length, 0.08, chains(B, T), [(b * 3) % (T + 1) for b in range(B)])


@pytest.mark.parametrize("T,H,dtype,latent,rope", [(1, 1, HF, 512, 64), (1, 16, BF, 512, 64), (1, 128, BF, 256, 32), (16, 16, HF, 128, 64)])
def test_one_long_sequence(T, H, dtype, latent, rope):
    cache, table = make(14, [41003], T, 64, latent, rope, dtype)
    check(normal(10, 1, T, H, latent + rope, dtype=dtype), cache, table, [41003], 0.07, chains(1, T))


def test_slots_past_32_bit_offsets():
    """Rows whose elements lie past 2^31 and whose bytes past 2^32."""
    n, size = 66000, 64                                   # 4224000 rows of 576 elements: 2.4e9 elements
    rows = torch.empty(n, size, 576, dtype=BF, device="cuda")
    cache = lm.LatentCache(rows, 512)
    table = ints([[65999, 3, 65998, 60001, 59999]])
    for i, p in enumerate(table[0].tolist()):
        rows[p] = normal(i, size, 576, dtype=BF)
    check(normal(20, 1, 2, 16, 576, dtype=BF), cache, table, [290], 0.07)
    x, key = normal(21, 2, 512, dtype=BF), normal(22, 2, 64, dtype=BF)
    lm.fa_latent_write(cache, x, key, ints([65999 * 64 + 63, 60001 * 64]))
    assert torch.equal(rows[65999, 63], torch.cat([x[0], key[0]])) and torch.equal(rows[60001, 0], torch.cat([x[1], key[1]]))
    moved = rows[59999, 5].clone()
    lm.fa_latent_keep(cache, table, ints([192]), ints([[69, -1]]))
    assert torch.equal(rows[60001, 0], moved)


def test_captured_twice_and_on_another_stream():
    """Two graphs with a workspace each, replayed side by side on lengths that change."""
    cache, table = make(15, [500] * 6, 2, 16, 512, 64, BF)
    q = normal(11, 6, 2, 20, 576, dtype=BF)
    mask = chains(6, 2)
    length = [ints([500, 20, 0, 130, 499, 64]), ints([1, 2, 3, 440, 5, 6])]
    attends = [lm.LatentAttention(6, 2, 20, 512, 64, BF) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    attends[0](q, cache, table, length[0], 0.07, mask)
    torch.cuda.synchronize()
    graphs = []
    for a, n in zip(attends, length):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            a(q, cache, table, n, 0.07, mask)
    for turn in range(3):
        for n in length:
            n.copy_((n + 37 * turn) % 500)
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for a, n in zip(attends, length):
            got = a.out.clone(), a.lse.clone()
            want = check(q, cache, table, n.tolist(), 0.07, mask)
            assert all(torch.equal(x, y) for x, y in zip(got, want))
    other = lm.LatentAttention(6, 2, 20, 512, 64, BF)
    got = other(q, cache, table, length[0], 0.07, mask, stream=streams[0])
    streams[0].synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, check(q, cache, table, length[0].tolist(), 0.07, mask)))


def test_refusals_of_the_binding():
    cache, table = make(16, [50], 1, 16, 128, 16, HF)
    q = normal(8, 1, 1, 4, 144, dtype=HF)
    attend = lm.LatentAttention(1, 1, 4, 128, 16, HF)
    for bad, error in ((q.to(BF), TypeError), (q[..., :128], ValueError), (q.cpu(), TypeError)):
        with pytest.raises(error):
            attend(bad, cache, table, ints([50]), 0.1)
    with pytest.raises(ValueError):
        attend(q, lm.LatentCache(cache.rows, 0), table, ints([50]), 0.1)
    with pytest.raises(ValueError):
        lm.LatentAttention(1, 1, 4, 256, 16, HF)(normal(1, 1, 1, 4, 272, dtype=HF), cache, table, ints([50]), 0.1)
    with pytest.raises(Exception):
        attend(q, cache, table, ints([50]), 0.0)


@pytest.mark.parametrize("dtype,latent,rope,size,length,T,H", [
    (BF, 512, 64, 64, [61000, 47003, 20, 15001], 3, 64),
    (HF, 512, 64, 16, [119000, 0, 1], 2, 128),
    (BF, 512, 16, 4, [40001, 90003], 5, 67),
    (BF, 384, 32, 128, [100000, 71777], 1, 1000),
    (HF, 256, 32, 64, [250001], 3, 80),
    (BF, 256, 32, 256, [150000, 99999], 1, 200),
    (HF, 128, 16, 32, [300000, 199999], 2, 99)])
def test_more_slots_than_the_cache_keeps(dtype, latent, rope, size, length, T, H):
    """Caches of 128 MiB and more: many tiles a run, 3 to 16 blocks of rows, whole and ragged, a page that is not held."""
    cache, table = make(T, length, T, size, latent, rope, dtype)
    table[0, 3] = -1
    B = len(length)
    count = [max(T - b, 0) for b in range(B)]
    q = normal(H, B, T, H, latent + rope, dtype=dtype)
    out, lse = check(q, cache, table, length, 0.06, chains(B, T), count)
    again = lm.LatentAttention(B, T, H, latent, rope, dtype)(q, cache, table, ints(length), 0.06, chains(B, T), ints(count))
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])
    check(q, cache, table, [min(n, 9000) for n in length], 0.06, chains(B, T))
