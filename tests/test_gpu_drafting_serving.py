"""Draft and verify over a latent cache, with tokens drawn at random and with a pool of pages that runs out: pages, slots,
writes, attention, verification and the moves of the accepted path as a program uses them together."""
import pytest

torch = pytest.importorskip("torch")

from constrained_decoding_diffusion_gb300 import drafting, lm, native, synth  # noqa: E402

pytestmark = pytest.mark.gpu


def rotate(x, pos, dim):
    w = 10000.0 ** (-torch.arange(0, dim, 2, dtype=torch.float64, device="cuda") / dim)
    z = torch.polar(torch.ones(pos.numel(), dim // 2, dtype=torch.float64, device="cuda"), pos.double()[:, None] * w)
    z = z.view(pos.numel(), *[1] * (x.dim() - 2), dim // 2)
    y = torch.complex(x[..., :dim // 2], x[..., dim // 2:]) * z
    return torch.cat((y.real, y.imag), -1)


def setup(B, seed=0, states=12, vocab=60, latent=True):
    fa = synth.random_dfa(states, vocab, 0.5, 2, 3)
    aut = native.fa_compile(fa)
    layer = drafting.LatentLayer.random(vocab, 64, 4, 128, 32, seed=seed) if latent else drafting.Layer.random(vocab, 64, 4, 2, 32, seed=seed)
    nxt, _ = lm.fa_beam_tables(aut)
    first = (nxt[int(fa.start)] >= 0).nonzero()[:, 0]
    return fa, aut, layer, nxt, first[torch.arange(B, device="cuda") % first.numel()]


def guesses(V, depth, seed=7):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return lambda pending: torch.log_softmax(3 * torch.randn((pending.shape[0], depth, V), generator=g, device="cuda"), -1)


@pytest.mark.parametrize("beams,depth", [(1, 1), (4, 3), (3, 5)])
def test_kept_tokens_are_the_choices_of_a_latent_layer(beams, depth):
    """By 64-bit logits from the cached vectors, up to the attention's error: weights and results in bf16 put an
    element off by at most (2^-8 + 2^-8 + 2^-9) sum_t p |c| (the scores' own error, 2^-17 of a few tens, is inside the last
    term), so two logits differ by at most twice that times |head|."""
    B = 3
    fa, aut, layer, nxt, first = setup(B, beams)
    run = drafting.Drafting(aut, layer, first, int(fa.start), beams, depth, max_length=40, page_size=8)
    rounds = 0
    drafter = guesses(fa.vocab, depth)
    while bool((run.pending >= 0).any()):
        run.round(drafter)
        rounds += 1
        assert rounds <= 40
    text = torch.cat(run.text, 1)
    table = nxt.cpu().numpy().astype(int)
    L, H = 128, 4
    for b in range(B):
        tokens = text[b][text[b] >= 0].long()
        n = tokens.numel()
        assert n == int(run.length[b]) and int(run.pages.held[b]) == -(-n // 8)
        pos = torch.arange(n, device="cuda")
        cached = run.cache.rows[run.table[b, pos // 8].long(), pos % 8].double()
        x = layer.embed[tokens]
        want = (x @ layer.down).double()
        want = torch.cat((want[:, :L], rotate(want[:, L:], pos, 32)), -1)
        assert ((cached - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -14 * want.abs().amax(-1, keepdim=True)).all()
        q = torch.einsum("te,ehd->thd", x, layer.wq)
        q = torch.cat((q[..., :L].double(), rotate(q[..., L:].double(), pos, 32).to(torch.bfloat16).double()), -1)
        s = torch.einsum("thd,sd->ths", q, cached) * 160 ** -0.5
        s = s.masked_fill(pos[None, None] > pos[:, None, None], -torch.inf)
        p = torch.softmax(s, -1)
        out = torch.einsum("ths,sd->thd", p, cached[:, :L]).reshape(n, H * L)
        off = torch.einsum("ths,sd->thd", p, cached[:, :L].abs()).reshape(n, H * L) * (2.0 ** -7 + 2.0 ** -9)
        logits, err = out @ layer.head.double(), off @ layer.head.double().abs()
        state = int(fa.start)
        for t in range(n):
            token = int(tokens[t])
            if t:
                live = torch.from_numpy(table[state] >= 0).cuda()
                best = torch.where(live, logits[t - 1] - err[t - 1], -torch.inf).max()
                assert live[token] and logits[t - 1, token] + err[t - 1, token] >= best
            state = table[state, token]
            assert state >= 0
    run.release()
    assert int(run.pages.n_free) == run.pages.free.shape[0]


@pytest.mark.parametrize("latent", [False, True])
def test_drawn_tokens_have_the_layers_distribution(latent):
    """The token after the first one, over 4000 sequences that start alike: frequencies within 5 sqrt(p (1 - p) / n) of
    the layer's own distribution under the automaton, which every sequence computes alike."""
    B, depth = 4000, 2
    fa, aut, layer, nxt, first = setup(B, 5, vocab=40, latent=latent)
    first = first[:1].expand(B).contiguous()
    seen = {}

    class Watched(drafting.Drafting):
        def logits(self, tokens, count):
            x = super().logits(tokens, count)
            seen.setdefault("p", torch.softmax(x[0, 0].double() / self.temperature, -1))
            return x
    run = Watched(aut, layer, first, int(fa.start), 3, depth, max_length=8, page_size=4, generator=torch.Generator(device="cuda").manual_seed(3),
                  temperature=1.5)
    state = int(run.state[0])
    got = run.round(guesses(fa.vocab, depth))
    second = torch.where(got[:, 1] >= 0, got[:, 1], run.pending)
    live = nxt[state] >= 0
    assert live[second.long()].all()
    p = torch.where(live, seen["p"], 0.0)
    p /= p.sum()
    have = torch.bincount(second.long(), minlength=fa.vocab).double() / B
    assert ((have - p).abs() <= 5 * (p * (1 - p) / B).sqrt() + 1e-9).all()
    rounds = 1
    while bool((run.pending >= 0).any()):
        run.round(guesses(fa.vocab, depth, rounds))
        rounds += 1
        assert rounds <= 8
    table = nxt.cpu().numpy().astype(int)
    for row in torch.cat(run.text, 1)[:50].cpu().tolist():
        state = int(fa.start)
        for token in (x for x in row if x >= 0):
            state = table[state, token]
            assert state >= 0
    run.release()
    assert int(run.pages.n_free) == run.pages.free.shape[0]


@pytest.mark.parametrize("latent", [False, True])
def test_a_pool_that_runs_out_only_delays(latent):
    """With room for some drafts at a time the other sequences sit rounds out, and the text is the same.  A text of up to 24
    tokens holds 6 pages and a draft of 7 takes 2 more: 38 pages serve six texts and one draft."""
    B, depth = 6, 3
    fa, aut, layer, nxt, first = setup(B, 9, latent=latent)
    texts, rounds = [], []
    for n_pages in (None, 38):
        run = drafting.Drafting(aut, layer, first, int(fa.start), 2, depth, max_length=24, page_size=4, n_pages=n_pages,
                                cache_dtype=torch.bfloat16)
        n = 0
        drafter = guesses(fa.vocab, depth)
        while bool((run.pending >= 0).any()):
            run.round(drafter)
            run.release()
            n += 1
            assert n <= 400
        text = torch.cat(run.text, 1).cpu()
        texts.append([row[row >= 0].tolist() for row in text])
        rounds.append(n)
    assert [t[:20] for t in texts[0]] == [t[:20] for t in texts[1]]
    assert rounds[1] > rounds[0]
