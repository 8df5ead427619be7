"""Draft and verify under an automaton: the model-side operators run together.

A drafter gives the log-probabilities of the next `depth` positions at once, as a diffusion model's
block does.  Beams over them that stay inside the automaton become a tree of drafted tokens, one
attention layer verifies the whole tree in a single pass over its paged cache, and the longest path
that agrees with the layer's own choices is kept.  The text is that of choosing one token at a time,
the best one or a random one; the draft only decides how many come from one pass.  The sequences share a
pool of pages: each has those that its text takes, and for the length of a pass those of its draft (or, of a pool
with room for all, those of its longest text from the start).

    python -m constrained_decoding_diffusion_gb300.drafting
"""
from __future__ import annotations

from typing import NamedTuple

import torch

from . import lm, native, synth


class Layer(NamedTuple):
    """One attention layer between an embedding and a vocabulary: embed [V, E], wq [E, H, D],
    wk, wv [E, KV, D] in a 16-bit type, and head [H * D, V] in float32."""
    embed: torch.Tensor
    wq: torch.Tensor
    wk: torch.Tensor
    wv: torch.Tensor
    head: torch.Tensor

    @classmethod
    def random(cls, vocab: int, width: int, heads: int, kv_heads: int, dim: int, seed: int = 0, dtype=torch.bfloat16):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def made(*shape, fan):
            return torch.randn(shape, generator=g, device="cuda") * fan ** -0.5
        return cls(made(vocab, width, fan=1).to(dtype), made(width, heads, dim, fan=width).to(dtype),
                   made(width, kv_heads, dim, fan=width).to(dtype), made(width, kv_heads, dim, fan=width).to(dtype),
                   4 * made(heads * dim, vocab, fan=heads * dim))


class LatentLayer(NamedTuple):
    """The same with one latent vector a token for all heads, in absorbed form: embed [V, E], wq [E, H, L + R] and
    down [E, L + R] in a 16-bit type, and head [H * L, V] in float32.  The last R elements carry the positions."""
    embed: torch.Tensor
    wq: torch.Tensor
    down: torch.Tensor
    head: torch.Tensor

    @classmethod
    def random(cls, vocab: int, width: int, heads: int, latent: int, rope: int, seed: int = 0, dtype=torch.bfloat16):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def made(*shape, fan):
            return torch.randn(shape, generator=g, device="cuda") * fan ** -0.5
        return cls(made(vocab, width, fan=1).to(dtype), made(width, heads, latent + rope, fan=width).to(dtype),
                   made(width, latent + rope, fan=width).to(dtype), 4 * made(heads * latent, vocab, fan=heads * latent))

    @property
    def latent_dim(self) -> int:
        return self.head.shape[0] // self.wq.shape[1]


class Drafting:
    """The text of B sequences under a DFA.  `pending` [B] is each sequence's next token, chosen but
    not yet in the cache (-1: the sequence has ended), `state` [B] the automaton's state after it.

    With a generator tokens are drawn from the softmax of the layer's logits / temperature under the automaton,
    else the best one is taken.  cache_dtype is that of the keys and values, float8_e4m3fn by default; a latent cache has its
    layer's type.  n_pages is the size of the pool (enough for all sequences and their drafts by
    default): a sequence whose draft finds no pages sits the round out (`waits` [B]).  Texts keep their pages until
    release(), so the pool must hold all of them and one draft, or a round comes in which nobody moves: stuck() says so, and
    release() may help where some texts have ended."""

    def __init__(self, aut: native.CompiledAutomaton, layer, first, start_state: int, beams: int = 4, depth: int = 4,
                 max_length: int = 1024, page_size: int = 16, cache_dtype=None, n_pages=None, generator=None,
                 temperature: float = 1.0):
        B, K = first.shape[0], beams
        (V, _), (_, H, D) = layer.embed.shape, layer.wq.shape
        self.latent = isinstance(layer, LatentLayer)
        if self.latent and cache_dtype not in (None, layer.wq.dtype):
            raise TypeError("a latent cache has its layer's type, %s, not %s" % (layer.wq.dtype, cache_dtype))
        if depth < 1 or 1 + K * depth > lm.FA_MAX_DRAFT:
            raise ValueError("beams * depth must be in [1, %d)" % lm.FA_MAX_DRAFT)
        self.layer, self.beams, self.depth, self.max_length = layer, K, depth, max_length
        T = 1 + K * depth                                  # the pending token, then the beams, one after another
        if n_pages is not None and n_pages * page_size < T:
            raise ValueError("a pool of %d pages of %d slots cannot hold a draft of %d tokens" % (n_pages, page_size, T))
        per = -(-(max_length + T) // page_size)
        i32 = dict(dtype=torch.int32, device="cuda")
        self._pages = lm.PageTables.empty(B, per, B * per if n_pages is None else n_pages, page_size)
        self.table, n_pages = self._pages.table, self._pages.free.shape[0]
        self.length = torch.zeros(B, **i32)
        self.dealt = n_pages >= B * per
        if self.dealt:                                     # room for every text and its draft: no round need ask for pages
            lm.fa_pages_resize(self._pages, torch.full((B,), per * page_size, **i32))
        if self.latent:
            L = layer.latent_dim
            self.cache = lm.LatentCache.empty(n_pages, page_size, L, D - L, layer.wq.dtype)
            self.attend = lm.LatentAttention(B, T, H, L, D - L, layer.wq.dtype)
            self.drafted = torch.full((B,), T, **i32)
        else:
            KV = layer.wk.shape[1]
            self.cache = lm.KVCache.empty(n_pages, KV, page_size, D, torch.float8_e4m3fn if cache_dtype is None else cache_dtype)
            self.attend = lm.TreeAttention(B, T, H, KV, D, layer.wq.dtype)
        self.phase, _ = lm.rope_phases(D - L if self.latent else D)
        self.next, self.live = lm.fa_beam_tables(aut)
        node = torch.arange(T, **i32)
        parents = torch.where((node - 1) % depth == 0, 0, node - 1)
        parents[0] = -1
        self.parents = parents.expand(B, T).contiguous()
        self.mask, self.below = lm.fa_tree_mask(self.parents)
        self.first_beam = lm.BeamSelect(B, 1, V, K)
        self.more_beams = lm.BeamSelect(B, K, V, K)
        self.generator, self.temperature = generator, temperature
        if generator is not None:
            self.accept = lm.Verify(B, T, V)
        else:
            self.choose = lm.BeamSelect(B * T, 1, V, 1)
            self.nothing = torch.zeros((B * T, 1), device="cuda")
        self.pending = first.to(**i32)
        self.state = self._move(torch.full((B,), start_state, **i32), self.pending)
        self.waits = self.moved = torch.zeros(B, dtype=torch.bool, device="cuda")   # of the last round
        self.text = []                                     # [B, at most 1 + depth] of each round, -1 where there is none

    @property
    def pages(self) -> lm.PageTables:
        """The pool, and the pages that each text takes.  A pool with room for everything is dealt out at the start; from the
        first look at it on, pages go round by round, as from a smaller one."""
        if self.dealt:
            self.dealt = False
            lm.fa_pages_resize(self._pages, self.length)
        return self._pages

    def _move(self, state, token):
        """The automaton's next state, -1 from and by -1."""
        to = self.next[state.clamp(min=0).long(), token.clamp(min=0).long()].int()
        return torch.where((state >= 0) & (token >= 0), to, -1)

    def draft(self, logp):
        """The best beams [B, K, depth] over logp [B, depth, V] from the automaton's current states."""
        B, K = self.pending.shape[0], self.beams
        hist = torch.full((B, 1, self.depth), -1, dtype=torch.int32, device="cuda")
        scores, states = torch.zeros((B, 1), device="cuda"), self.state.view(B, 1)
        for t in range(self.depth):
            select = self.more_beams if t else self.first_beam
            # every beam reads the position's one row
            scores, parent, token, states = select(logp[:, t:t + 1].expand(B, hist.shape[1], -1), scores, states, self.next, self.live)
            hist = lm.fa_beam_reorder(hist, parent, token=token, at=t)
        return hist

    def logits(self, tokens, count):
        """The layer's logits [B, T, V] after the drafted tokens [B, T], of which count [B] are in use; their keys
        and values join the cache."""
        B, T = tokens.shape
        positions = self.length.view(B, 1) + self.below
        x = self.layer.embed[tokens.clamp(min=0).long()]
        if self.latent:
            L, scale = self.layer.latent_dim, self.layer.wq.shape[2] ** -0.5
            q = torch.einsum("bte,ehd->bthd", x, self.layer.wq)
            turned = q.view(B * T, *q.shape[2:])[..., L:]
            lm.fa_rope(turned, positions.view(-1), self.phase, out=turned)
            down = (x @ self.layer.down).view(B * T, -1)
            slot, _, _, _ = lm.fa_slot_map(self._pages, self.length, self.drafted, B * T)
            lm.fa_latent_write(self.cache, down[:, :L], down[:, L:], slot, positions.view(-1), self.phase)
            out, _ = self.attend(q, self.cache, self.table, self.length, scale, self.mask, count)
        else:
            q, k, v = (torch.einsum("bte,ehd->bthd", x, w) for w in self.layer[1:4])
            lm.fa_rope(q.view(B * T, *q.shape[2:]), positions.view(-1), self.phase, out=q.view(B * T, *q.shape[2:]))
            lm.fa_cache_write(self.cache, k, v, self.table, self.length, count, positions, self.phase)
            out, _ = self.attend(q, self.cache, self.table, self.length, self.mask, count)
        return out.float().view(B, T, -1) @ self.layer.head

    def best(self, logits, tokens, hist):
        """The longest path of drafted tokens that are the best ones, and what follows: (path, token, state)."""
        B, K, depth = hist.shape
        T = tokens.shape[1]
        # the automaton's state at every node, and the layer's choice there
        state = torch.empty((B, K, depth), dtype=torch.int32, device="cuda")
        for t in range(depth):
            state[:, :, t] = self._move(state[:, :, t - 1] if t else self.state.view(B, 1).expand(B, K), hist[:, :, t])
        state = torch.cat((self.state.view(B, 1), state.view(B, K * depth)), 1)
        logp = torch.log_softmax(logits, -1)
        _, _, want, after = self.choose(logp.view(B * T, 1, -1), self.nothing, state.view(B * T, 1).contiguous(), self.next, self.live)
        want, after = want.view(B, T), after.view(B, T)
        # a beam's tokens are kept while each is the choice at the node before
        node = 1 + torch.arange(K * depth, device="cuda").view(1, K, depth).expand(B, K, depth)
        before = torch.where(torch.arange(depth, device="cuda") > 0, node - 1, 0)
        same = (hist >= 0) & (hist == want.gather(1, before.reshape(B, -1)).view(B, K, depth))
        kept, beam = same.int().cumprod(-1).sum(-1).max(1)
        path = torch.where(torch.arange(depth, device="cuda") < kept.view(B, 1), 1 + beam.view(B, 1) * depth + torch.arange(depth, device="cuda"), -1)
        path = torch.cat((torch.zeros((B, 1), dtype=path.dtype, device="cuda"), path), 1)
        last = path.max(1, keepdim=True).values
        return path, want.gather(1, last).view(B), after.gather(1, last).view(B)

    def drawn(self, logits, tokens, count):
        """The same with tokens drawn at random: the draft is kept as far as the draws agree with it."""
        u = torch.rand(tokens.shape, generator=self.generator, device="cuda")
        path, _, token, state = self.accept(torch.softmax(logits / self.temperature, -1), tokens, self.parents, u, count=count,
                                            states=self.state, next=self.next, live=self.live)
        return path[:, :1 + self.depth], token, state

    def verify(self, hist):
        """One pass over the tree; returns the tokens that join the text [B, 1 + depth]."""
        B, K, depth = hist.shape
        tokens = torch.cat((self.pending.view(B, 1), hist.view(B, K * depth)), 1)
        T = tokens.shape[1]
        alive = self.pending >= 0
        if not self.dealt:
            room = lm.fa_pages_resize(self._pages, self.length + T * alive.int()) == lm.FA_PAGES_OK
            self.waits = alive & ~room
            alive &= room
        self.moved = alive
        count = torch.where(alive, T, 0).int()
        logits = self.logits(tokens, count)
        path, token, after = self.best(logits, tokens, hist) if self.generator is None else self.drawn(logits, tokens, count)
        path = torch.where(alive.view(B, 1), path, -1).int()
        (lm.fa_latent_keep if self.latent else lm.fa_cache_keep)(self.cache, self.table, self.length, path)
        joined = torch.where(path >= 0, tokens.gather(1, path.clamp(min=0).long()), -1)
        self.length += (path >= 0).sum(1).int()
        if not self.dealt:
            lm.fa_pages_resize(self._pages, self.length)
        done = alive & (self.length >= self.max_length)
        self.state = torch.where(done, -1, torch.where(alive, after, self.state))
        self.pending = torch.where(done, -1, torch.where(alive, token, self.pending))
        self.text.append(joined)
        return joined

    def release(self):
        """The pages of sequences that have ended go back to the pool, and their texts leave the cache."""
        self.length = torch.where(self.pending >= 0, self.length, 0)
        if not self.dealt:
            lm.fa_pages_resize(self._pages, self.length)

    def stuck(self) -> bool:
        """Whether the last round moved nobody for want of pages, so that the next one will not either unless pages are
        released (reads the device)."""
        return bool(self.waits.any() & ~self.moved.any())

    def round(self, drafter):
        """drafter(pending [B]) -> log-probabilities [B, depth, V] of the positions after pending."""
        return self.verify(self.draft(drafter(self.pending)))


def main():
    fa = synth.random_dfa(64, 1000, 0.5, 8, 1)
    aut = native.fa_compile(fa)
    layer = Layer.random(fa.vocab, 256, 8, 2, 64)
    B, depth = 8, 4
    guess = torch.randn((256, depth, fa.vocab), generator=torch.Generator(device="cuda").manual_seed(2), device="cuda") / 16

    def drafter(pending):
        x = layer.embed[pending.clamp(min=0).long()].float()
        return torch.log_softmax(torch.einsum("be,edv->bdv", x, guess), -1)
    nxt, _ = lm.fa_beam_tables(aut)
    first = (nxt[int(fa.start)] >= 0).nonzero()[:B, 0]
    run = Drafting(aut, layer, first, int(fa.start), depth=depth, max_length=200)
    rounds = 0
    while bool((run.pending >= 0).any()) and rounds < 200:
        run.round(drafter)
        if run.stuck():
            raise SystemExit("the pool holds none of the drafts that are left")
        rounds += 1
    print("%d rounds, lengths %s" % (rounds, run.length.tolist()))


if __name__ == "__main__":
    main()
