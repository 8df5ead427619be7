"""The serving operators at the ends of their sizes: many sequences, long drafts, many rows, large vocabularies.
Tolerances as in the operators' own tests."""
import random

import pytest

torch = pytest.importorskip("torch")

import serving_reference as ref  # noqa: E402
from constrained_decoding_diffusion_gb300 import lm  # noqa: E402
from test_gpu_latent import BF, HF, chains, check, ints, make, normal  # noqa: E402

pytestmark = pytest.mark.gpu


def test_attention_of_very_many_rows():
    """1024 drafted tokens of 60 heads: 960 blocks of rows of one sequence, and of one with 3 tokens in use."""
    cache, table = make(1, [130, 70], 1024, 64, 128, 16, BF)
    check(normal(2, 2, 1024, 60, 144, dtype=BF), cache, table, [130, 70], 0.08, chains(2, 1024), [1024, 3])


def test_attention_of_1024_heads():
    cache, table = make(3, [200, 0, 65], 1, 8, 128, 32, HF)
    check(normal(4, 3, 1, 1024, 160, dtype=HF), cache, table, [200, 0, 65], 0.08)


def test_attention_of_thousands_of_sequences():
    B = 5000
    length = [b % 7 for b in range(B)]
    cache, table = make(5, length, 1, 8, 128, 16, BF)
    check(normal(6, B, 1, 2, 144, dtype=BF), cache, table, length, 0.08)


def test_a_table_that_could_hold_two_billion_slots():
    """Only the lengths say what is read of a table; a length past it ends with it."""
    page, per = 1024, (2 ** 31 - 8192) // 1024
    cache = lm.LatentCache(normal(7, 3, page, 144, dtype=BF), 128)
    table = torch.full((1, per), -1, dtype=torch.int32, device="cuda")
    table[0, :2] = ints([2, 0])
    q = normal(8, 1, 1, 16, 144, dtype=BF)
    attend = lm.LatentAttention(1, 1, 16, 128, 16, BF)
    small = lm.LatentAttention(1, 1, 16, 128, 16, BF)
    for n in (1500, 2047):
        got = [x.clone() for x in attend(q, cache, table, ints([n]), 0.08)]
        want = small(q, cache, table[:, :3].contiguous(), ints([n]), 0.08)
        assert all(torch.equal(x, y) for x, y in zip(got, want))


@pytest.mark.parametrize("V", [9_999_991, 24_000_000])
@pytest.mark.parametrize("draft", [True, False])
def test_verification_over_millions_of_tokens(V, draft):
    g = torch.Generator(device="cuda").manual_seed(V)
    target = torch.softmax(4 * torch.randn(1, 3, V, generator=g, device="cuda"), -1)
    q = torch.softmax(4 * torch.randn(1, 3, V, generator=g, device="cuda"), -1) if draft else None
    best = target[0, 0].topk(2).indices
    d = dict(target=target, tokens=torch.stack((best[0] * 0, best[0], best[1]))[None].int(),
             parents=ints([[-1, 0, 0]]), u=torch.tensor([[0.73, 0.4, 0.6]], device="cuda"), draft=q)
    got = lm.Verify(1, 3, V)(**d)
    want = ref.verify(target, d["tokens"], d["parents"], d["u"], q)
    assert all((x.cpu().numpy() == y).all() for x, y in zip(got[:3], want))


def test_verification_of_many_sequences():
    B, V = 20000, 3
    g = torch.Generator().manual_seed(1)
    target = torch.rand(B, 3, V, generator=g).cuda()
    d = dict(target=target, tokens=torch.randint(0, V, (B, 3), generator=g).int().cuda(), parents=ints([[-1, 0, 1]] * B),
             u=torch.rand(B, 3, generator=g).cuda(), draft=torch.rand(B, 3, V, generator=g).cuda())
    got = lm.Verify(B, 3, V)(**d)
    want = ref.verify(target, d["tokens"], d["parents"], d["u"], d["draft"])
    assert all((x.cpu().numpy() == y).all() for x, y in zip(got[:3], want))


def test_pages_and_slots_of_65535_sequences():
    B, per, size = 65535, 3, 4
    rng = random.Random(5)
    pages = lm.PageTables.empty(B, per, 120000, size)
    pool = ref.Pool(pages)
    for _ in range(3):
        want = [rng.randint(0, 13) for _ in range(B)]
        status = lm.fa_pages_resize(pages, ints(want))
        assert status.cpu().tolist() == pool.resize(want)
        pool.same(pages)
    start, count = [rng.randint(0, 5) for _ in range(B)], [rng.randint(0, 6) for _ in range(B)]
    got = lm.fa_slot_map(pages, ints(start), ints(count), 190000)
    for g, w in zip(got, ref.slot_map(pool.table, 120000, size, start, count, 190000)):
        assert g.cpu().tolist() == w


def test_a_table_of_many_pages():
    pages = lm.PageTables.empty(3, 400000, 1000000, 1)
    pool = ref.Pool(pages)
    for want in ([400000, 1, 399999], [5, 300000, 0], [400001, 0, 400000], [0, 400000, 400000]):
        assert lm.fa_pages_resize(pages, ints(want)).cpu().tolist() == pool.resize(want)
        pool.same(pages)


def test_many_tokens_written_and_a_long_path():
    cache = lm.LatentCache.empty(1500, 256, 128, 16, HF)
    N = 300001
    x, key = normal(1, N, 128, dtype=HF), normal(2, N, 16, dtype=HF)
    slot = torch.randperm(1500 * 256, generator=torch.Generator().manual_seed(1))[:N].int().cuda()
    lm.fa_latent_write(cache, x, key, slot)
    flat = cache.rows.view(-1, 144)
    assert torch.equal(flat[slot.long()], torch.cat([x, key], 1))
    path = torch.arange(0, 2048, 2, dtype=torch.int32, device="cuda")[None]
    table = torch.arange(1500, dtype=torch.int32, device="cuda")[None]
    want = flat[100:100 + 2048:2].clone()
    lm.fa_latent_keep(cache, table, ints([100]), path)
    # (as bits: some slots have never been written and may hold NaN)
    assert torch.equal(flat[100:100 + 1024].view(torch.int16), want.view(torch.int16))


def test_write_of_more_tokens_than_32_bits_count_threads():
    """The tokens share one vector (a stride of zero); the last ones' slots are written, and no other."""
    N = 2 ** 28 + 41
    cache = lm.LatentCache(torch.zeros(8, 16, 144, dtype=HF, device="cuda"), 128)
    x, key = normal(1, 1, 128, dtype=HF), normal(2, 1, 16, dtype=HF)
    slot = torch.full((N,), -1, dtype=torch.int32, device="cuda")
    slot[2 ** 28 - 1:] = torch.arange(3, 45, dtype=torch.int32, device="cuda")
    lm.fa_latent_write(cache, x.expand(N, 128), key.expand(N, 16), slot)
    want = torch.zeros(128, 144, dtype=HF, device="cuda")
    want[3:45] = torch.cat([x, key], 1)
    assert torch.equal(cache.rows.view(128, 144), want)
