"""The model-side operators where a call spans many blocks: one call must give the very bits of the
same work in pieces (every vector is worked out alone), and beams in 16-bit types must follow the
automaton at any alignment."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import lm_reference as ref  # noqa: E402
from constrained_decoding_diffusion_gb300 import lm, native, synth  # noqa: E402

pytestmark = pytest.mark.gpu

BF, HF, FP, F8 = torch.bfloat16, torch.float16, torch.float32, torch.float8_e4m3fn


def randn(seed, *shape, dtype=FP):
    return torch.randn(shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").to(dtype)


@pytest.mark.parametrize("dtype", [FP, HF, BF])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("heads,dim,rot", [(5, 64, 64), (3, 128, 32), (1, 1024, 1024)])
def test_rope_of_many_tokens(dtype, interleaved, heads, dim, rot):
    n = 20011
    x = randn(1, n, heads, dim, dtype=dtype)
    pos = torch.randint(0, 1 << 20, (n,), dtype=torch.int32, device="cuda")
    phase, _ = lm.rope_phases(rot)
    whole = lm.fa_rope(x, pos, phase, interleaved=interleaved)
    parts = [lm.fa_rope(x[i:i + 777], pos[i:i + 777], phase, interleaved=interleaved) for i in range(0, n, 777)]
    assert torch.equal(whole, torch.cat(parts))


@pytest.mark.parametrize("dtype", [FP, HF, BF])
@pytest.mark.parametrize("fmt", [HF, F8])
@pytest.mark.parametrize("heads,dim,rot", [(3, 128, 128), (7, 48, 16), (2, 256, 64)])
def test_cache_write_of_many_tokens(dtype, fmt, heads, dim, rot):
    B, T, page = 3, 7001, 64
    per = -(-T // page)
    table = torch.randperm(B * per, generator=torch.Generator().manual_seed(2))[:B * per].int().view(B, per).cuda()
    k, v = randn(1, B, T, heads, dim, dtype=dtype), randn(2, B, T, heads, dim, dtype=dtype)
    k[1, 5000, 1, 3] = float("nan")
    v[2, 17, 0] = 0.0
    pos = torch.randint(0, 1 << 20, (B, T), dtype=torch.int32, device="cuda")
    phase, _ = lm.rope_phases(rot)
    got = []
    for step in (T, 613):
        cache = lm.KVCache.empty(B * per, heads, page, dim, fmt)
        for x in cache:
            if x is not None:
                x.view(torch.uint8).zero_()
        for i in range(0, T, step):
            start = torch.full((B,), i, dtype=torch.int32, device="cuda")
            lm.fa_cache_write(cache, k[:, i:i + step], v[:, i:i + step], table, start, positions=pos[:, i:i + step].contiguous(), phase=phase)
        got.append([x.view(torch.uint8) for x in cache if x is not None])
    assert all(torch.equal(x, y) for x, y in zip(*got))


@pytest.mark.parametrize("dtype", [HF, BF, FP])
@pytest.mark.parametrize("V,top", [(50, 3), (3001, 40), (8195, 256), (30003, 16)])
@pytest.mark.parametrize("pad", [0, 1, 3])
def test_beams_of_unaligned_rows_under_an_automaton(dtype, V, top, pad):
    fa = synth.random_dfa(24, V, 0.7, 6, V)
    nxt, live = lm.fa_beam_tables(native.fa_compile(fa))
    N, K = 3, 5
    logp = (randn(V, N, K, V + pad) * 2).log_softmax(-1).to(dtype)[..., pad:]
    scores = -3 * torch.rand((N, K), device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))
    states = torch.randint(0, fa.n_states, (N, K), dtype=torch.int32, device="cuda", generator=torch.Generator(device="cuda").manual_seed(2))
    got = lm.BeamSelect(N, K, V, top, dtype)(logp, scores, states, nxt, live)
    want = ref.beam(logp, scores, top, states.cpu().numpy(), nxt.cpu().numpy())
    for g, w in zip(got, want):
        assert np.array_equal(g.cpu().numpy(), w)
