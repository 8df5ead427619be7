"""What Drafting refuses before it touches the device (CPU only)."""
import pytest

torch = pytest.importorskip("torch")

from constrained_decoding_diffusion_gb300 import drafting  # noqa: E402


def latent_layer(dtype=torch.bfloat16):
    return drafting.LatentLayer(*(torch.zeros(shape, dtype=dtype) for shape in ((40, 64), (64, 4, 160), (64, 160))), torch.zeros(512, 40))


@pytest.mark.parametrize("dtype,cache", [(torch.bfloat16, torch.float8_e4m3fn), (torch.bfloat16, torch.float16), (torch.float16, torch.bfloat16)])
def test_a_latent_cache_of_another_type(dtype, cache):
    with pytest.raises(TypeError, match="latent cache"):
        drafting.Drafting(None, latent_layer(dtype), torch.zeros(2, dtype=torch.int32), 0, cache_dtype=cache)


def test_a_pool_that_holds_no_draft():
    with pytest.raises(ValueError, match="draft of 13 tokens"):
        drafting.Drafting(None, latent_layer(), torch.zeros(2, dtype=torch.int32), 0, beams=4, depth=3, page_size=4, n_pages=3)
