"""Draft and verify under an automaton: the model-side operators run together.

A drafter gives the log-probabilities of the next `depth` positions at once, as a diffusion model's
block does.  Beams over them that stay inside the automaton become a tree of drafted tokens, one
attention layer verifies the whole tree in a single pass over its paged cache, and the longest path
that agrees with the layer's own choices is kept.  The text is that of choosing one token at a time;
the draft only decides how many come from one pass.

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


class Drafting:
    """The text of B sequences under a DFA.  `pending` [B] is each sequence's next token, chosen but
    not yet in the cache (-1: the sequence has ended), `state` [B] the automaton's state after it."""

    def __init__(self, aut: native.CompiledAutomaton, layer: Layer, first, start_state: int, beams: int = 4, depth: int = 4,
                 max_length: int = 1024, page_size: int = 16, cache_dtype=torch.float8_e4m3fn):
        B, K = first.shape[0], beams
        (V, _), (_, H, D), KV = layer.embed.shape, layer.wq.shape, layer.wk.shape[1]
        if depth < 1 or 1 + K * depth > lm.FA_MAX_DRAFT:
            raise ValueError("beams * depth must be in [1, %d)" % lm.FA_MAX_DRAFT)
        self.layer, self.beams, self.depth, self.max_length = layer, K, depth, max_length
        T = 1 + K * depth                                  # the pending token, then the beams, one after another
        per = -(-(max_length + T) // page_size)
        i32 = dict(dtype=torch.int32, device="cuda")
        self.cache = lm.KVCache.empty(B * per, KV, page_size, D, cache_dtype)
        self.table = torch.arange(B * per, **i32).view(B, per)
        self.length = torch.zeros(B, **i32)
        self.phase, _ = lm.rope_phases(D)
        self.next, self.live = lm.fa_beam_tables(aut)
        node = torch.arange(T, **i32)
        parents = torch.where((node - 1) % depth == 0, 0, node - 1)
        parents[0] = -1
        self.mask, self.below = lm.fa_tree_mask(parents.expand(B, T).contiguous())
        self.attend = lm.TreeAttention(B, T, H, KV, D, layer.wq.dtype)
        self.first_beam = lm.BeamSelect(B, 1, V, K)
        self.more_beams = lm.BeamSelect(B, K, V, K)
        self.choose = lm.BeamSelect(B * T, 1, V, 1)
        self.nothing = torch.zeros((B * T, 1), device="cuda")
        self.pending = first.to(**i32)
        self.state = self._move(torch.full((B,), start_state, **i32), self.pending)
        self.text = []                                     # [B, at most 1 + depth] of each round, -1 where there is none

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

    def verify(self, hist):
        """One pass over the tree; returns the tokens that join the text [B, 1 + depth]."""
        B, K, depth = hist.shape
        tokens = torch.cat((self.pending.view(B, 1), hist.view(B, K * depth)), 1)
        T = tokens.shape[1]
        count = torch.where(self.pending >= 0, T, 0).int()
        positions = self.length.view(B, 1) + self.below
        x = self.layer.embed[tokens.clamp(min=0).long()]
        q, k, v = (torch.einsum("bte,ehd->bthd", x, w) for w in self.layer[1:4])
        lm.fa_rope(q.view(B * T, *q.shape[2:]), positions.view(-1), self.phase, out=q.view(B * T, *q.shape[2:]))
        lm.fa_cache_write(self.cache, k, v, self.table, self.length, count, positions, self.phase)
        out, _ = self.attend(q, self.cache, self.table, self.length, self.mask, count)
        logp = torch.log_softmax(out.float().view(B, T, -1) @ self.layer.head, -1)
        # the automaton's state at every node, and the layer's choice there
        state = torch.empty((B, K, depth), dtype=torch.int32, device="cuda")
        for t in range(depth):
            state[:, :, t] = self._move(state[:, :, t - 1] if t else self.state.view(B, 1).expand(B, K), hist[:, :, t])
        state = torch.cat((self.state.view(B, 1), state.view(B, K * depth)), 1)
        _, _, want, after = self.choose(logp.view(B * T, 1, -1), self.nothing, state.view(B * T, 1).contiguous(), self.next, self.live)
        want, after = want.view(B, T), after.view(B, T)
        # a beam's tokens are kept while each is the choice at the node before
        node = 1 + torch.arange(K * depth, device="cuda").view(1, K, depth).expand(B, K, depth)
        before = torch.where(torch.arange(depth, device="cuda") > 0, node - 1, 0)
        same = (hist >= 0) & (hist == want.gather(1, before.reshape(B, -1)).view(B, K, depth))
        kept, beam = same.int().cumprod(-1).sum(-1).max(1)
        path = torch.where(torch.arange(depth, device="cuda") < kept.view(B, 1), 1 + beam.view(B, 1) * depth + torch.arange(depth, device="cuda"), -1)
        path = torch.cat((torch.zeros((B, 1), dtype=path.dtype, device="cuda"), path), 1)
        path = torch.where(self.pending.view(B, 1) >= 0, path, -1).int()
        lm.fa_cache_keep(self.cache, self.table, self.length, path)
        joined = torch.where(path >= 0, tokens.gather(1, path.clamp(min=0).long()), -1)
        last = path.max(1, keepdim=True).values.clamp(min=0).long()
        alive = self.pending >= 0
        self.length += (path >= 0).sum(1).int()
        alive &= self.length < self.max_length
        self.state = torch.where(alive, after.gather(1, last).view(B), -1)
        self.pending = torch.where(alive, want.gather(1, last).view(B), -1)
        self.text.append(joined)
        return joined

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
        rounds += 1
    print("%d rounds, lengths %s" % (rounds, run.length.tolist()))


if __name__ == "__main__":
    main()
