"""Draft and verify with a pool that is too small: the caller learns of it."""
import pytest

torch = pytest.importorskip("torch")

from constrained_decoding_diffusion_gb300 import drafting  # noqa: E402
from test_gpu_drafting_serving import guesses, setup  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("latent", [False, True])
def test_a_pool_too_small_for_all_texts_is_noticed(latent):
    """Six texts of up to 24 tokens take 36 pages of 4 and a draft of 7 two more; with 20 pages a round comes in which nobody
    moves.  The loop ends there rather than spin, every text is intact, and waits names those that have no pages."""
    B, depth = 6, 3
    fa, aut, layer, nxt, first = setup(B, 9, latent=latent)
    texts = {}
    for n_pages in (None, 20):
        run = drafting.Drafting(aut, layer, first, int(fa.start), 2, depth, max_length=24, page_size=4, n_pages=n_pages,
                                cache_dtype=torch.bfloat16)
        assert not run.stuck()
        drafter = guesses(fa.vocab, depth)
        rounds = 0
        while bool((run.pending >= 0).any()):
            before = run.length.clone()
            run.round(drafter)
            moved = run.length > before
            assert torch.equal(run.moved, moved) and not bool((run.waits & moved).any())
            if run.stuck():
                break
            rounds += 1
            assert rounds <= 200
        texts[n_pages] = [row[row >= 0].tolist() for row in torch.cat(run.text, 1).cpu()]
        if n_pages is None:
            assert not run.stuck() and not bool(run.waits.any())
        else:
            assert run.stuck() and torch.equal(run.waits, run.pending >= 0)
    for whole, part in zip(texts[None], texts[20]):
        assert whole[:len(part)][:20] == part[:20] and len(part) < 24 + 4


@pytest.mark.parametrize("seed", range(4))
def test_release_helps_where_texts_have_ended(seed):
    """Two texts of up to 24 tokens and 14 pages of 4.  A text that has not ended holds 6 pages at most and its next draft of 7
    takes it to 8, so the first one is only held up by a second one that has ended (7 pages at most), or the other way
    round: release() helps every time."""
    fa, aut, layer, nxt, first = setup(2, seed)
    run = drafting.Drafting(aut, layer, first, int(fa.start), 2, 3, max_length=24, page_size=4, n_pages=14)
    drafter = guesses(fa.vocab, 3, seed)
    rounds = 0
    while bool((run.pending >= 0).any()):
        run.round(drafter)
        if run.stuck():
            assert bool((run.pending < 0).any())
            run.release()
            run.round(drafter)
            assert not run.stuck()
        rounds += 1
        assert rounds <= 100
