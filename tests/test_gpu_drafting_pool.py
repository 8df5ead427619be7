"""Draft and verify with a pool that has room for everything: it is dealt out once."""
import pytest

torch = pytest.importorskip("torch")

from constrained_decoding_diffusion_gb300 import drafting, lm  # noqa: E402
from test_gpu_drafting_serving import guesses, setup  # noqa: E402

pytestmark = pytest.mark.gpu


def texts(run, drafter, look=None):
    rounds = 0
    while bool((run.pending >= 0).any()):
        if look is not None and rounds == look:
            pages = run.pages
            size, length = pages.page_size, run.length.tolist()
            assert pages.held.tolist() == [-(-n // size) for n in length]
            assert int(pages.n_free) == pages.free.shape[0] - int(pages.held.sum())
            for row, held in zip(pages.table.tolist(), pages.held.tolist()):
                assert min(row[:held], default=0) >= 0 and set(row[held:]) <= {-1}
        run.round(drafter)
        rounds += 1
        assert rounds <= 60
    return [row[row >= 0].tolist() for row in torch.cat(run.text, 1).cpu()], rounds


@pytest.mark.parametrize("latent", [False, True])
def test_no_round_asks_for_pages(latent, monkeypatch):
    """The calls of a loop over the default pool, and its texts against those of a loop that is looked at and so goes round by
    round, from the start or from the middle."""
    fa, aut, layer, nxt, first = setup(4, 3, latent=latent)
    calls = []
    resize = lm.fa_pages_resize
    monkeypatch.setattr(drafting.lm, "fa_pages_resize", lambda *a, **k: (calls.append(1), resize(*a, **k))[1])

    def loop(look):
        run = drafting.Drafting(aut, layer, first, int(fa.start), 2, 3, max_length=30, page_size=4)
        del calls[:]
        got = texts(run, guesses(fa.vocab, 3), look)
        n = len(calls)
        assert run.pages.held.tolist() == [-(-x // 4) for x in run.length.tolist()]
        run.release()
        assert int(run.pages.n_free) == run.pages.free.shape[0]
        return got, n
    (want, rounds), n = loop(None)
    assert n == 0
    for look in (0, 2):
        (got, again), n = loop(look)
        assert (got, again) == (want, rounds) and n == 1 + 2 * (rounds - look)


def test_release_before_a_look_and_pages_taken_by_the_caller():
    """Ended texts give their pages back at the first look, and what a caller takes out of the pool is missed."""
    fa, aut, layer, nxt, first = setup(4, 3)
    run = drafting.Drafting(aut, layer, first, int(fa.start), 2, 3, max_length=12, page_size=4)
    run.round(guesses(fa.vocab, 3))
    run.pending[1:] = -1
    run.release()
    assert run.length[1:].tolist() == [0, 0, 0] and int(run.length[0]) > 0
    pages = run.pages
    assert pages.held.tolist() == [-(-int(run.length[0]) // 4), 0, 0, 0]
    left = int(pages.n_free)
    pages.n_free.zero_()                                       # the caller has them all
    run.round(guesses(fa.vocab, 3))
    assert run.stuck() and run.waits.tolist() == [True, False, False, False]
    pages.n_free.fill_(left)
    run.round(guesses(fa.vocab, 3))
    assert not run.stuck() and run.moved.tolist() == [True, False, False, False]
