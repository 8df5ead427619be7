"""Beam selection refuses outputs over inputs except in place (CPU only; the pointers are never followed)."""
import pytest

from test_lm_refusals import P, lib, refused  # noqa: F401

STEP = 1 << 16


def select(lib, N=2, K=4, top=4, **at):  # noqa: F811
    names = ("scores", "states", "score", "parent", "token", "state")
    a = {name: P + (i + 2) * STEP for i, name in enumerate(names)}
    for name, (other, by) in at.items():
        a[name] = a[other] + by
    return lib.fa_beam_select(0, N, K, 100, top, P, 400, 100, a["scores"], a["states"], 5, P + STEP, P + STEP, a["score"], a["parent"],
                              a["token"], a["state"], P, 1 << 30, None)


@pytest.mark.parametrize("kw", [dict(state=("states", 4)), dict(state=("states", -4)), dict(score=("scores", 16)),
                                dict(parent=("scores", 0)), dict(token=("states", 0)), dict(state=("scores", 0)),
                                dict(score=("states", 0)), dict(K=8, state=("states", 0)), dict(K=2, score=("scores", 0))])
def test_beam_select_over_its_inputs(lib, kw):  # noqa: F811
    refused(lib, select(lib, **kw))
