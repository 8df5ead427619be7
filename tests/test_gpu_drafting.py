"""Draft and verify: what is kept is what choosing one token at a time from the same cache gives.

A kept token must be the best live one by 64-bit logits from the cached keys and values, up to
the attention's error.  With weights in bf16 (fp16 for an 8-bit cache) and bf16 outputs, an output
element is off by at most (2^-8 + 2^-9 + 2^-9) sum_t p |v| here (scores below 16: their own error,
2^-17 of a few tens, is inside the last term), so two logits differ by at most twice that times |head|."""
import pytest

torch = pytest.importorskip("torch")

from constrained_decoding_diffusion_gb300 import drafting, lm, native, synth  # noqa: E402

pytestmark = pytest.mark.gpu


def rotate(x, pos, dim):
    w = 10000.0 ** (-torch.arange(0, dim, 2, dtype=torch.float64, device="cuda") / dim)
    z = torch.polar(torch.ones(pos.numel(), dim // 2, dtype=torch.float64, device="cuda"), pos.double()[:, None] * w)[:, None]
    y = torch.complex(x[..., :dim // 2], x[..., dim // 2:]) * z
    return torch.cat((y.real, y.imag), -1)


@pytest.mark.parametrize("cache_dtype", [torch.bfloat16, torch.float8_e4m3fn])
@pytest.mark.parametrize("beams,depth,good", [(1, 1, False), (4, 3, True), (5, 6, False), (3, 4, True)])
def test_kept_tokens_are_the_choices_of_the_layer(cache_dtype, beams, depth, good):
    fa = synth.random_dfa(12, 60, 0.5, 2, 3)
    aut = native.fa_compile(fa)
    B, E, H, KV, D = 3, 64, 4, 2, 32
    layer = drafting.Layer.random(fa.vocab, E, H, KV, D, seed=beams)
    nxt, _ = lm.fa_beam_tables(aut)
    first = (nxt[int(fa.start)] >= 0).nonzero()[:B, 0]
    run = drafting.Drafting(aut, layer, first, int(fa.start), beams, depth, max_length=40, page_size=8, cache_dtype=cache_dtype)
    g = torch.Generator(device="cuda").manual_seed(7)
    truth = drafting.Drafting(aut, layer, first, int(fa.start), 1, 1, max_length=60, page_size=8, cache_dtype=cache_dtype)
    flat = torch.zeros((B, 1, fa.vocab), device="cuda")
    while truth.length.max() < 50:
        truth.round(lambda pending: flat)
    ahead = torch.cat(truth.text, 1).cpu()
    ahead = [row[row >= 0].tolist() for row in ahead]

    def drafter(pending):
        logp = torch.randn((B, depth, fa.vocab), generator=g, device="cuda")
        if good:                                           # the text that choosing one at a time gave, mostly
            for b in range(B):
                n = int(run.length[b])
                for t in range(depth):
                    if n + 1 + t < len(ahead[b]) and t != 2:
                        logp[b, t, ahead[b][n + 1 + t]] += 20.0
        return torch.log_softmax(logp, -1)
    rounds = 0
    while bool((run.pending >= 0).any()):
        before = run.length.clone()
        got = run.round(drafter)
        assert ((got >= 0).sum(1) == run.length - before).all()
        rounds += 1
        assert rounds <= 40
    text = torch.cat(run.text, 1)
    n_max = int(run.length.max())
    k, v = (torch.empty((B, n_max, KV, D), dtype=torch.float32, device="cuda") for _ in range(2))
    lm.fa_cache_read(run.cache, run.table, run.length, k, v)
    table = nxt.cpu().numpy().astype(int)
    total = 0
    for b in range(B):
        tokens = text[b][text[b] >= 0].long()
        n = tokens.numel()
        assert n == int(run.length[b])
        total += n
        x = layer.embed[tokens]
        pos = torch.arange(n, device="cuda")
        # the cache holds the kept tokens' keys and values: 2^-8 of a rounding, or half a step of e4m3
        want_k = rotate(torch.einsum("te,ehd->thd", x, layer.wk).double(), pos, D)
        want_v = torch.einsum("te,ehd->thd", x, layer.wv).double()
        for have, want in ((k, want_k), (v, want_v)):
            top = want.abs().amax(-1, keepdim=True)
            u = 2.0 ** -8 if cache_dtype == torch.bfloat16 else 2.0 ** -4
            assert ((have[b, :n].double() - want).abs() <= u * want.abs() + 2.0 ** -6 * u * top).all()
        q = rotate(torch.einsum("te,ehd->thd", x, layer.wq).double(), pos, D)
        q = q.to(torch.bfloat16).double().view(n, KV, H // KV, D)
        kd, vd = k[b, :n].double(), v[b, :n].double()
        s = torch.einsum("tkgd,skd->tkgs", q, kd) * D ** -0.5
        s = s.masked_fill(pos[None, None, None] > pos[:, None, None, None], -torch.inf)
        p = torch.softmax(s, -1)
        out = torch.einsum("tkgs,skd->tkgd", p, vd).reshape(n, H * D)
        off = torch.einsum("tkgs,skd->tkgd", p, vd.abs()).reshape(n, H * D) * 2.0 ** -7
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
    if good:
        assert rounds < total / B / 1.5                    # more than one token of a pass is kept


def test_example_runs(capsys):
    drafting.main()
    assert "rounds" in capsys.readouterr().out


def test_refusals():
    fa = synth.real_number_dfa()
    aut = native.fa_compile(fa)
    layer = drafting.Layer.random(fa.vocab, 32, 2, 1, 16)
    with pytest.raises(ValueError):
        drafting.Drafting(aut, layer, torch.zeros(1, dtype=torch.int32, device="cuda"), 0, beams=64, depth=16)
