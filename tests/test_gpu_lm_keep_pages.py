"""Keeping an accepted path across pages that are missing: a slot without a page reads as zeros, is not
written, and the rest of the path moves all the same."""
import pytest

torch = pytest.importorskip("torch")

from constrained_decoding_diffusion_gb300 import lm  # noqa: E402

pytestmark = pytest.mark.gpu


def bits(x):
    return x.view({1: torch.uint8, 2: torch.int16, 4: torch.int32}[x.element_size()])


@pytest.mark.parametrize("fmt", [torch.bfloat16, torch.float8_e4m3fn])
@pytest.mark.parametrize("missing", [[], [0], [1], [2], [1, 3], [5], [7]])
def test_missing_pages(fmt, missing):
    page, per, n = 4, 6, 3
    cache = lm.KVCache.empty(2 * per, 2, page, 32, fmt)
    g = torch.Generator().manual_seed(1)
    for x in cache:
        if x is not None:
            bits(x).copy_(torch.randint(1, 100, x.shape, generator=g))
    table = torch.randperm(2 * per, generator=g).int().view(1, 2 * per)[:, :per].contiguous()
    for p in missing:
        if p < per:
            table[0, p] = -1 if p % 2 else 2 * per
    path = torch.tensor([[0, 2, 3, 5, 8, 9, 13, 16, 18, 30, -1, 40]], dtype=torch.int32)   # 30 lies past the table
    if 7 in missing:
        path[0, 9] = 17                                # does not ascend: ends the path
    was = [None if x is None else bits(x).cpu().clone() for x in cache]
    want = [None if x is None else x.clone() for x in was]
    for i, j in enumerate(path[0].tolist()):
        if j < 0 or (i and j <= path[0, i - 1]):
            break
        to, fr = n + i, n + j
        if int(table[0, to // page]) not in range(2 * per):
            continue
        held = fr // page < per and int(table[0, fr // page]) in range(2 * per)
        for x, y in zip(want, was):
            if x is not None:
                x[int(table[0, to // page]), :, to % page] = y[int(table[0, fr // page]), :, fr % page] if held else 0
    lm.fa_cache_keep(cache, table.cuda(), torch.tensor([n], dtype=torch.int32).cuda(), path.cuda())
    for x, y in zip(cache, want):
        if x is not None:
            assert torch.equal(bits(x).cpu(), y)
