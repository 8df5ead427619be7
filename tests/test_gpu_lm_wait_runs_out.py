"""A wait inside the tensor-core attention that runs out: the rows its block has a part in come out as NaN, all
others are right, and the next call is unaffected."""
import pytest

torch = pytest.importorskip("torch")

from constrained_decoding_diffusion_gb300 import lm, native  # noqa: E402
from test_gpu_lm_attention import F8, make, queries  # noqa: E402

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


@pytest.mark.parametrize("fmt,dtype,page", [(BF, BF, 64), (BF, BF, 4), (HF, HF, 16), (F8, BF, 16), (F8, HF, 256)])
@pytest.mark.parametrize("T,group", [(20, 1), (12, 4), (100, 1), (60, 4)])
@pytest.mark.parametrize("length", [[3000] * 9, [(37 * b) % 300 for b in range(500)]])
def test_rows_of_the_first_block(fmt, dtype, page, T, group, length):
    B, kv = len(length), 2
    cache, table = make(T, length, T, kv, page, 64, fmt)
    q = queries(T, B, T, kv * group, 64, dtype=dtype)
    n = torch.tensor(length, dtype=torch.int32).cuda()
    attend = lm.TreeAttention(B, T, kv * group, kv, 64, dtype)
    clean, lse = (x.clone() for x in attend(q, cache, table, n))
    assert torch.isfinite(clean).all()
    native.fa_debug_inject_wait_timeouts(1)
    try:
        out, l2 = (x.clone() for x in attend(q, cache, table, n))
    finally:
        native.fa_debug_inject_wait_timeouts(0)
    lost = torch.isnan(l2)
    assert torch.equal(lost, torch.isnan(out).all(-1)) and torch.equal(lost, torch.isnan(out).any(-1))
    assert torch.equal(out[~lost], clean[~lost]) and torch.equal(l2[~lost], lse[~lost])
    # the block takes the first units of the list: whole ones, in the order of sequences and heads
    units = lost.view(B, T, kv, group).permute(0, 2, 1, 3).reshape(B * kv, T * group)
    some, first = units.any(1), int(units.any(1).sum())
    assert 1 <= first < B * kv and some[:first].all() and units[:first].all()
    out, l2 = attend(q, cache, table, n)
    assert torch.equal(out, clean) and torch.equal(l2, lse)
