"""What the phase table's maker refuses (CPU)."""
import math

import pytest

torch = pytest.importorskip("torch")

from constrained_decoding_diffusion_gb300 import lm  # noqa: E402


@pytest.mark.parametrize("kw", [dict(rot_dim=3), dict(rot_dim=-2), dict(scaling="other"), dict(factor=0.5), dict(base=0.0),
                                dict(scaling="blend", fast_turns=1.0), dict(scaling="blend", fast_turns=1.0, slow_turns=4.0),
                                dict(factor=math.nan), dict(base=math.nan), dict(factor=math.inf), dict(base=math.inf),
                                dict(scaling="blend", fast_turns=math.nan), dict(scaling="blend", slow_turns=math.nan)])
def test_refusals(kw):
    with pytest.raises(ValueError):
        lm.rope_phases(**{"rot_dim": 16, "device": "cpu", **kw})


def test_turns_do_not_matter_without_a_blend():
    a, m = lm.rope_phases(16, fast_turns=1.0, slow_turns=1.0, device="cpu")
    b, n = lm.rope_phases(16, device="cpu")
    assert torch.equal(a, b) and m == n == 1.0
