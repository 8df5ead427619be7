"""Queries whose dimensions of one element have strides that mean nothing."""
import pytest

torch = pytest.importorskip("torch")

from constrained_decoding_diffusion_gb300 import lm  # noqa: E402
from test_gpu_lm_attention import F8, make, queries  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,T,H", [(1, 1, 1), (3, 1, 2), (1, 30, 2), (2, 5, 1)])
def test_single_elements(B, T, H):
    dim, length = 64, [70, 3, 150][:B]
    cache, table = make(1, length, T, 1, 16, dim, F8)
    n = torch.tensor(length, dtype=torch.int32).cuda()
    q = queries(2, B, T, H, dim, dtype=torch.bfloat16)
    attend = lm.TreeAttention(B, T, H, 1, dim)
    want = [x.clone() for x in attend(q, cache, table, n)]
    odd = q.as_strided(q.shape, [1 if size == 1 else by for size, by in zip(q.shape, q.stride())])
    assert 1 in odd.stride()[:3]
    assert all(torch.equal(x, y) for x, y in zip(attend(odd, cache, table, n), want))
