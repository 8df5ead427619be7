"""Beam selection in a loop that hands a call's scores and states to the next one: they lie where its
results go, and every result must still follow its parent's old state."""
import pytest

torch = pytest.importorskip("torch")

from constrained_decoding_diffusion_gb300 import lm, native, synth  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("N,K,V", [(1, 64, 300), (3, 64, 1501), (2, 256, 300), (5, 33, 20011), (200, 40, 100), (700, 64, 50)])
def test_outputs_given_back_as_inputs(N, K, V):
    fa = synth.random_dfa(97, V, 0.7, 9, V)
    nxt, live = lm.fa_beam_tables(native.fa_compile(fa))
    g = torch.Generator(device="cuda").manual_seed(K)
    scores = -torch.rand((N, K), generator=g, device="cuda")
    states = torch.randint(0, fa.n_states, (N, K), generator=g, dtype=torch.int32, device="cuda")
    looped, apart = (lm.BeamSelect(N, K, V, K) for _ in range(2))
    kept = (scores, states)
    for _ in range(8):
        logp = torch.randn((N, K, V), generator=g, device="cuda").log_softmax(-1)
        # few live tokens in a step: slots past the last cell get the state -1
        logp[:, :, 40:] = torch.where(torch.rand((N, 1, 1), generator=g, device="cuda") < 0.3, -torch.inf, logp[:, :, 40:])
        want = [x.clone() for x in apart(logp, *kept, nxt, live)]
        kept = (want[0].clone(), want[3].clone())
        got = looped(logp, scores, states, nxt, live)
        scores, _, _, states = got
        for x, y in zip(got, want):
            assert torch.equal(x, y)
        up, token = want[1].clamp(min=0).long(), want[2].clamp(min=0).long()
        assert (want[1] >= 0).any() and up.max() < K and token.max() < V


def test_one_sequence_grows_in_place():
    """N = 1 with fewer beams in than out: the inputs are the first of the outputs' places."""
    fa = synth.random_dfa(31, 500, 0.7, 9, 2)
    nxt, live = lm.fa_beam_tables(native.fa_compile(fa))
    select = lm.BeamSelect(1, 32, 500, 200)
    logp = torch.randn((1, 32, 500), generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").log_softmax(-1)
    start = torch.arange(32, dtype=torch.int32, device="cuda").view(1, 32) % 31
    want = [x.clone() for x in select(logp, torch.zeros((1, 32), device="cuda"), start, nxt, live)]
    select.score[:, :32], select.state[:, :32] = 0.0, start
    got = select(logp, select.score[:, :32], select.state[:, :32], nxt, live)
    assert all(torch.equal(x, y) for x, y in zip(got, want))
