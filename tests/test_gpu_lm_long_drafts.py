"""Drafts of hundreds of tokens, as a prompt's or a long block's: more than two row blocks of 256, mask words
beyond the fourth, up to the limit of 1024."""
import pytest

torch = pytest.importorskip("torch")

from constrained_decoding_diffusion_gb300 import lm  # noqa: E402
from test_gpu_lm_attention import F8, check, make, queries  # noqa: E402

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


class Masked:
    """TreeAttention with the mask words of a given matrix in place of the chain's."""

    def __init__(self, B, T, H, kv, dim, dtype, seen):
        self.attend = lm.TreeAttention(B, T, H, kv, dim, dtype)
        self.out, self.lse = self.attend.out, self.attend.lse
        words = (T + 63) // 64
        bits = torch.zeros((B, T, words * 64), dtype=torch.int64, device="cuda")
        bits[..., :T] = seen
        place = torch.arange(64, device="cuda")
        self.mask = (bits.view(B, T, words, 64) << place).sum(-1)   # (bit 63 wraps to the sign)

    def __call__(self, q, cache, table, length, mask, count):
        return self.attend(q, cache, table, length, self.mask, count)


@pytest.mark.parametrize("fmt,dtype,dim,page", [(BF, BF, 128, 64), (F8, BF, 64, 16), (HF, HF, 80, 128), (F8, HF, 128, 2)])
@pytest.mark.parametrize("T,group", [(500, 1), (257, 4), (1024, 1), (1024, 3)])
def test_chains(fmt, dtype, dim, page, T, group):
    length = [0, 1500, 77]
    cache, table = make(T, length, T, 2, page, dim, fmt, spread=1.0)
    q = queries(T, len(length), T, 2 * group, dim, dtype=dtype)
    check(q, cache, table, length)
    check(q, cache, table, length, count=[T, T - 1, 333 % T])


@pytest.mark.parametrize("fmt,dtype", [(BF, BF), (F8, BF)])
@pytest.mark.parametrize("T,group", [(500, 2), (1024, 1)])
def test_any_mask(fmt, dtype, T, group):
    """Rows that see a tenth of the draft, all of it, one token of the last word, or nothing of it."""
    length = [0, 300]
    cache, table = make(T + 1, length, T, 1, 16, 64, fmt)
    q = queries(T, 2, T, group, 64, dtype=dtype)
    g = torch.Generator(device="cuda").manual_seed(T)
    seen = torch.rand((2, T, T), generator=g, device="cuda") < 0.1
    seen[:, 3] = True
    seen[:, 4:9] = False
    seen[:, 6, T - 1] = True
    seen[:, 200:] &= torch.arange(T, device="cuda") >= 130       # tiles of the draft that no row of a block sees
    check(q, cache, table, length, seen=seen, attend=Masked(2, T, group, 1, 64, dtype, seen))
    check(q, cache, table, length, seen=seen, count=[T - 7, 64], attend=Masked(2, T, group, 1, 64, dtype, seen))
