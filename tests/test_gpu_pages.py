"""Pages handed out on the device and slots of a ragged batch, against Python lists.  All outputs are whole
numbers."""
import random

import pytest

torch = pytest.importorskip("torch")

import serving_reference as ref  # noqa: E402
from constrained_decoding_diffusion_gb300 import lm  # noqa: E402

pytestmark = pytest.mark.gpu


def ints(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


def resize(pages, pool, want):
    status = lm.fa_pages_resize(pages, ints(want))
    assert status.cpu().tolist() == pool.resize(want)
    pool.same(pages)


@pytest.mark.parametrize("B,per,n,size", [(1, 1, 1, 1), (1, 4, 3, 16), (5, 7, 20, 4), (33, 20, 300, 16), (1000, 9, 4000, 64),
                                          (1025, 5, 3000, 2), (3000, 40, 50000, 1024)])
def test_sequences_come_and_go(B, per, n, size):
    rng = random.Random(B)
    pages = lm.PageTables.empty(B, per, n, size)
    pool = ref.Pool(pages)
    for turn in range(12):
        most = size * per * (1.0 if turn % 3 else 1.1)
        want = [rng.choice([0, rng.randint(-3, int(most)), rng.randint(0, size), pool.held[b] * size]) for b in range(B)]
        resize(pages, pool, want)
    resize(pages, pool, [0] * B)
    assert int(pages.n_free) == n and sorted(pages.free.cpu().tolist()) == list(range(n))


def test_a_pool_that_runs_out():
    """The first sequence that does not fit, and every later one that grows, gets nothing; the others go on."""
    pages = lm.PageTables.empty(6, 10, 12, 8)
    pool = ref.Pool(pages)
    resize(pages, pool, [16, 8, 80, 0, 0, 0])      # 2 + 1 + 10 pages of 12
    resize(pages, pool, [16, 8, 72, 8, 8, 0])      # all but the last of the third's
    resize(pages, pool, [0, 8, 80, 8, 0, 8])       # what the first gives back serves the third
    resize(pages, pool, [2 ** 31 - 1, -2 ** 31, 81, 8, 0, 8])


def test_an_undone_call_restores_the_stack():
    pages = lm.PageTables.empty(40, 30, 700, 16)
    pool = ref.Pool(pages)
    rng = random.Random(1)
    a, b = [rng.randint(0, 250) for _ in range(40)], [rng.randint(0, 250) for _ in range(40)]
    resize(pages, pool, a)
    before = [x.clone() for x in pages[:4]]
    resize(pages, pool, b)
    resize(pages, pool, a)
    assert all(torch.equal(x, y) for x, y in zip(before, pages[:4]))


def test_no_pool_and_no_table():
    for per, n in ((0, 5), (5, 0)):
        pages = lm.PageTables.empty(3, per, n, 4)
        resize(pages, ref.Pool(pages), [0, 4, -1])


def test_counts_out_of_range_stay_inside_the_arrays():
    """held and n_free are taken as the nearest bound, and what lies around the arrays is left alone."""
    wide = torch.full((4 * 6 + 9 + 200,), 77, dtype=torch.int32, device="cuda")
    table, free = wide[100:124].view(4, 6), wide[130:139]
    table.fill_(3)
    free.fill_(5)
    for held, n_free, want in (([9, -4, 6, 100], 50, [0, 24, 0, 24]), ([100] * 4, 9, [0] * 4), ([-1] * 4, -5, [24] * 4),
                               ([0] * 4, 2 ** 31 - 1, [24, 12, 0, 0])):
        pages = lm.PageTables(table, ints(held), free, ints([n_free]), 4)
        lm.fa_pages_resize(pages, ints(want))
        assert 0 <= int(pages.n_free) <= 9 and ((pages.held >= 0) & (pages.held <= 6)).all()
        assert (wide[:100] == 77).all() and (wide[124:130] == 77).all() and (wide[139:] == 77).all()


@pytest.mark.parametrize("B,per,size,most", [(1, 3, 1, 3), (3, 5, 16, 40), (255, 6, 8, 30), (256, 6, 8, 30), (257, 4, 64, 100),
                                             (1300, 3, 2, 6), (7, 400, 16, 6000)])
def test_slots(B, per, size, most):
    rng = random.Random(B)
    n = B * per + 2
    pages = lm.PageTables(torch.randperm(n, generator=torch.Generator().manual_seed(B))[:B * per].int().view(B, per).cuda(),
                          None, torch.empty(n, dtype=torch.int32, device="cuda"), None, size)
    pages.table[B // 2, per // 2] = -1
    pages.table[0, 0] = n                                # no such page
    start = [rng.randint(-2, most) for _ in range(B)]
    count = [rng.choice([0, rng.randint(-1, most)]) for _ in range(B)]
    total = sum(max(c, 0) for c in count)
    table = pages.table.cpu().tolist()
    for N in sorted({0, 1, total // 2, total, total + 1, total + 1000}):
        got = lm.fa_slot_map(pages, ints(start), ints(count), N)
        for name, g, w in zip(("slot", "seq", "position", "offset"), got, ref.slot_map(table, n, size, start, count, N)):
            assert g.cpu().tolist() == w, (N, name)


def test_slots_of_no_sequence():
    pages = lm.PageTables.empty(0, 4, 5, 16)
    slot, seq, pos, offset = lm.fa_slot_map(pages, ints([]), ints([]), 3)
    assert slot.tolist() == seq.tolist() == pos.tolist() == [-1] * 3 and offset.tolist() == [0]


def test_counts_whose_sum_passes_32_bits():
    pages = lm.PageTables.empty(4, 2, 5, 16)
    slot, seq, pos, offset = lm.fa_slot_map(pages, ints([0] * 4), ints([5, 2 ** 31 - 1, 2 ** 31 - 1, 9]), 8)
    assert seq.tolist() == [0] * 5 + [1] * 3 and offset.tolist() == [0, 5, 8, 8, 8]


def test_captured():
    """A decoding step's pages in a graph: the lengths live on the device."""
    pages = lm.PageTables.empty(20, 12, 200, 4)
    pool = ref.Pool(pages)
    want, start, count = ints([0] * 20), ints([0] * 20), ints([1] * 20)
    status = torch.empty_like(want)
    lm.fa_pages_resize(pages, want)                      # loads the kernels
    out = lm.fa_slot_map(pages, start, count, 20)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lm.fa_pages_resize(pages, want, status)
        lm.fa_slot_map(pages, start, count, 20, out)
        start += 1
    for t in range(45):
        w = [t + 1 if (t + b) % 17 else 0 for b in range(20)]
        want.copy_(ints(w))
        graph.replay()
        assert status.cpu().tolist() == pool.resize(w)
        pool.same(pages)
        assert out[0].cpu().tolist() == ref.slot_map(pool.table, 200, 4, [t] * 20, [1] * 20, 20)[0]
