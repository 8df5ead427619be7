"""Results that a call makes on another stream do not take memory that the current stream may still use."""
import pytest

torch = pytest.importorskip("torch")

from constrained_decoding_diffusion_gb300 import lm, native, synth  # noqa: E402

pytestmark = pytest.mark.gpu


def free_block(n_bytes):
    """The address of a block that the current stream's memory has just got back, and would give out next."""
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    x = torch.empty(n_bytes, dtype=torch.uint8, device="cuda")
    at = x.data_ptr()
    del x
    probe = torch.empty(n_bytes, dtype=torch.uint8, device="cuda")
    assert probe.data_ptr() == at
    return at


def test_results_on_another_stream():
    side = torch.cuda.Stream()
    x = torch.randn((3001, 5, 128), device="cuda")
    pos = torch.arange(3001, dtype=torch.int32, device="cuda")
    phase, _ = lm.rope_phases(128)
    parents = torch.arange(-1, 999, dtype=torch.int32, device="cuda").expand(20, 1000).contiguous()
    src = torch.randint(0, 9, (30, 4, 10007), dtype=torch.int32, device="cuda")
    parent = torch.randint(-1, 4, (30, 4), dtype=torch.int32, device="cuda")
    aut = native.fa_compile(synth.random_dfa(64, 30011, 0.7, 8, 1))
    calls = [lambda s: (lm.fa_rope(x, pos, phase, stream=s),), lambda s: lm.fa_tree_mask(parents, stream=s),
             lambda s: (lm.fa_beam_reorder(src, parent, stream=s),), lambda s: lm.fa_beam_tables(aut, stream=s)]
    for call in calls:
        want = [y.clone() for y in call(None)]
        for i, y in enumerate(want):
            at = free_block(y.numel() * y.element_size())
            got = call(side)
            assert got[i].data_ptr() != at
            side.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, want))
            del got
