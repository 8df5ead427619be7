"""A phase table without pairs, as rope_phases(0) makes it: nothing is rotated."""
import pytest

torch = pytest.importorskip("torch")

from constrained_decoding_diffusion_gb300 import lm  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", [torch.bfloat16, torch.float8_e4m3fn])
@pytest.mark.parametrize("dim", [64, 67])
def test_keys_are_stored_as_they_are(fmt, dim):
    wide = torch.randn((2, 5, 3, dim), generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    k, v = wide[..., :64], wide.flip(0)[..., :64]
    pos = torch.arange(10, dtype=torch.int32, device="cuda").view(2, 5)
    table, start = torch.tensor([[0], [1]], dtype=torch.int32).cuda(), torch.zeros(2, dtype=torch.int32, device="cuda")
    got = []
    for more in ({}, dict(positions=pos, phase=lm.rope_phases(0)[0])):
        cache = lm.KVCache.empty(2, 3, 8, 64, fmt)
        for x in cache:
            if x is not None:
                x.view(torch.uint8).zero_()
        lm.fa_cache_write(cache, k, v, table, start, **more)
        got.append([x.view(torch.uint8) for x in cache if x is not None])
    assert all(torch.equal(x, y) for x, y in zip(*got))
    assert torch.equal(lm.fa_rope(k.reshape(10, 3, 64), pos.view(10), lm.rope_phases(0)[0]), k.reshape(10, 3, 64))
