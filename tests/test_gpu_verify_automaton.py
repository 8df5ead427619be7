"""Verification of a sampled draft under an automaton that its drafter need not know."""
import pytest

torch = pytest.importorskip("torch")

from constrained_decoding_diffusion_gb300 import lm  # noqa: E402
from test_gpu_verify import BF, F32, beams, chain, check, make  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("parents", [[-1, 0], [-1, 0, 0, 1]])
def test_first_and_second_token_have_the_targets_distribution(parents, masked):
    """Children drawn from the draft's row as given, or from its allowed tokens alone.  Of n draws each frequency of the
    token after node 0 is within 5 sqrt(p (1 - p) / n), and of those that kept token 1 the next one's likewise."""
    n, V = 60000, 6
    g = torch.Generator().manual_seed(2)
    p = torch.tensor([0.3, 0.05, 0.2, 0.25, 0.1, 0.1])
    q = torch.tensor([0.05, 0.3, 0.3, 0.05, 0.1, 0.2])
    nxt = torch.zeros(2, V, dtype=torch.int16)
    nxt[0, 2], nxt[0, 1], nxt[1, 0] = -1, 1, -1
    T = len(parents)
    tokens = torch.zeros(n, T, dtype=torch.int32)
    dead = torch.zeros(n, dtype=torch.long)                # the automaton's state at node 0
    for j in range(1, T):
        state = dead if parents[j] == 0 else nxt[0, tokens[:, parents[j]].long()].long().clamp(min=0)
        row = q.expand(n, V) * (nxt[state] >= 0) if masked else q.expand(n, V)
        tokens[:, j] = torch.multinomial(row, 1, generator=g)[:, 0].int()
    d = dict(target=p.expand(n, T, V).cuda(), tokens=tokens.cuda(), parents=torch.tensor([parents] * n, dtype=torch.int32).cuda(),
             u=torch.rand(n, T, generator=g).cuda(), draft=q.expand(n, T, V).cuda(), next=nxt.cuda(),
             live=((nxt >= 0).long() << torch.arange(V)).sum(-1, keepdim=True).int().cuda(),
             states=torch.zeros(n, dtype=torch.int32, device="cuda"))
    path, kept, token, _ = (x.cpu() for x in lm.Verify(n, T, V)(**d))
    first = torch.where(kept > 1, tokens.gather(1, path[:, 1:2].clamp(min=0).long())[:, 0], token).long()

    def same(have, state):
        want = torch.where(nxt[state] >= 0, p, 0.0)
        want /= want.sum()
        seen = torch.bincount(have, minlength=V) / have.numel()
        assert ((seen - want).abs() <= 5 * (want * (1 - want) / have.numel()).sqrt() + 1e-12).all()
    same(first, 0)
    one = (kept > 1) & (first == 1)
    second = torch.where(kept > 2, tokens.gather(1, path[:, -1:].clamp(min=0).long() if T < 3 else path[:, 2:3].clamp(min=0).long())[:, 0], token)
    same(second[one].long(), 1)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("draft", [True, False])
@pytest.mark.parametrize("V", [33, 5000, 98304])
def test_children_that_are_not_allowed_change_nothing(V, draft, dtype):
    """The same outputs, to the bit, as with such tokens taken out of the draft."""
    for parents in (chain(5), beams(3, 3), [-1] + [0] * 40):
        d = make(V + len(parents), 6, parents, V, dtype, draft, states=5, spread=1.5)
        want = check(d)
        state = [d["states"].long()]
        tokens = d["tokens"].clone()
        for j, p in enumerate(parents):
            if p >= 0:
                to = torch.where(state[p] >= 0, d["next"][state[p].clamp(min=0), tokens[:, j].long().clamp(min=0)].long(), -1)
                state.append(to)
                d["tokens"][:, j] = torch.where(to < 0, -1, tokens[:, j])
        assert (d["tokens"] != tokens).any()
        assert all(torch.equal(x, y) for x, y in zip(check(d), want))


def test_a_draft_row_with_weight_only_on_tokens_that_are_not_allowed():
    """As a row without weight: a child has q(x) = 0, and is accepted where the target has weight."""
    d = make(4, 4, [-1, 0, 0], 50, states=3)
    d["draft"] = torch.where(d["next"][d["states"].long()][:, None] < 0, d["draft"], 0.0)
    alive = [(d["next"][int(s)] >= 0).nonzero()[:, 0] for s in d["states"]]
    d["tokens"][:, 2] = torch.stack([x[0] for x in alive]).int()
    d["tokens"][:, 1] = torch.stack([(d["next"][int(s)] < 0).nonzero()[0, 0] for s in d["states"]]).int()
    path, kept, _, _ = check(d)
    assert (kept == 2).all() and (path[:, 1] == 2).all()
