"""The 64-bit reference of verification gives the target's distribution, whatever the draft knew."""
import pytest

torch = pytest.importorskip("torch")

import numpy as np  # noqa: E402

import serving_reference as ref  # noqa: E402


@pytest.mark.parametrize("children", [1, 2])
@pytest.mark.parametrize("masked", [False, True])
def test_a_sampled_draft_under_an_automaton(masked, children):
    """Target (.5, .5, dead), children drawn from (.4, .1, .5 dead) as given or from its allowed part: of n draws each
    frequency is within 5 sqrt(p (1 - p) / n) of (.5, .5, 0)."""
    n = 20000
    g = torch.Generator().manual_seed(children)
    p, q = torch.tensor([0.5, 0.5, 0.3]), torch.tensor([0.4, 0.1, 0.5])
    tokens = torch.multinomial((q * torch.tensor([1, 1, 1 - int(masked)])).expand(n, 3), 1 + children, replacement=True, generator=g).int()
    path, kept, token, _ = ref.verify(
        p.expand(n, 1 + children, 3), tokens, torch.tensor([[-1] + [0] * children] * n), torch.rand(n, 1 + children, generator=g),
        q.expand(n, 1 + children, 3), None, torch.zeros(n, dtype=torch.int32), torch.tensor([[0, 0, -1]], dtype=torch.int16))
    first = np.where(kept > 1, np.take_along_axis(tokens.numpy(), path[:, 1:2].clip(0), 1)[:, 0], token)
    seen = np.bincount(first, minlength=3) / n
    assert (abs(seen - [0.5, 0.5, 0.0]) <= [5 * (0.25 / n) ** 0.5] * 2 + [0]).all()
