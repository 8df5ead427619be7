"""The bits of verification's sums: draws next to a border between two tokens."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from constrained_decoding_diffusion_gb300 import lm  # noqa: E402
from test_gpu_serving_sizes import ints  # noqa: E402

pytestmark = pytest.mark.gpu


def split_row(V, sign, seed):
    """Log-normal weights of which the first half weighs sign 2^-42 of the sum more than the second: the prefix to the
    middle lies sign 2^-43 of the sum from a half of it.  The first weights of a half make up the difference, up to four floats of
    24 bits each; what that leaves is below 2^-60 of the sum.  fsum rounds once."""
    g = np.random.default_rng(seed)
    w = np.exp(4 * g.standard_normal(V)).astype(np.float32)
    half = V // 2
    w[:4] = w[half + 1:half + 5] = w[V - 1] = 0.0
    w[half - 1] = w[half] = 1.0
    a, c = math.fsum(w[:half].tolist()), math.fsum(w[half:].tolist())
    e = sign * 2.0 ** -42
    more = (e * (a + c) - (a - c)) / (1 - e)                   # that the first half lacks
    at = 0
    if more < 0:
        more, at = (a - c - e * (a + c)) / (1 + e), half + 1   # that the second one lacks
    for i in range(4):
        w[at + i] = np.float32(more)
        more -= float(w[at + i])
        if more < 0:                                           # rounded up: one step less, and the rest next
            more += float(w[at + i])
            w[at + i] = np.nextafter(w[at + i], np.float32(0))
            more -= float(w[at + i])
    a, c = math.fsum(w[:half].tolist()), math.fsum(w[half:].tolist())
    assert abs((a - c) / (a + c) - e) < 2.0 ** -50
    return w, half - 1 if sign > 0 else half


@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("V", [151936, 10_000_000, 24_000_000])
def test_a_draw_next_to_a_border(V, sign):
    """u = 1/2 and a border 2^-43 of the sum away: eight times what 46 bits of a sum leave.  By the target's sums alone, by
    those beside a draft's, and by those of a rejection (whose draft weighs nothing elsewhere)."""
    w, want = split_row(V, sign, V + sign)
    target = torch.from_numpy(w).cuda().view(1, 1, V).expand(1, 2, V)
    half = torch.full((1, 2), 0.5, device="cuda")
    call = lm.Verify(1, 2, V)

    def drawn(tokens, draft, row):
        path, kept, token, _ = call(row, ints([tokens]), ints([[-1, 0]]), half, draft=draft)
        assert kept.tolist() == [1]
        return token.tolist()
    assert drawn([0, -1], None, target) == [want]
    draft = torch.rand(1, 2, V, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))
    assert drawn([0, -1], draft, target) == [want]
    draft.zero_()
    draft[..., V - 1] = 1.0                                    # its token weighs nothing in the target: rejected, l = the sum
    assert drawn([0, V - 1], draft, target) == [want]
