"""Plain 64-bit implementations of verification, pages, slots and the latent cache, from their
definitions.  They share nothing with the package."""
from __future__ import annotations

import math

import numpy as np
import torch

HALF_ULP = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 2.0 ** -149, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}


def weights(x):
    x = x.double().cpu().numpy().copy()
    x[~((x > 0) & (x < np.inf))] = 0.0
    return x


def verify(target, tokens, parents, u, draft=None, count=None, states=None, next_state=None):
    """(path, kept, token, state), with the distributions themselves."""
    B, T, V = target.shape
    p = weights(target)
    q = None if draft is None else weights(draft)
    tok, par, uu = tokens.cpu().numpy(), parents.cpu().numpy(), u.double().cpu().numpy()
    path, kept = np.full((B, T), -1, np.int32), np.zeros(B, np.int32)
    token, state = np.full(B, -1, np.int32), np.full(B, -1, np.int32)
    nxt = None if next_state is None else next_state.cpu().numpy()
    for b in range(B):
        use = T if count is None else min(max(int(count[b]), 0), T)
        if use == 0:
            continue
        s = 0 if states is None else int(states[b])

        def allowed():
            if states is None:
                return np.ones(V, bool)
            return nxt[s] >= 0 if 0 <= s < nxt.shape[0] else np.zeros(V, bool)

        def spread(row):
            row = np.where(allowed(), row, 0.0)
            return row / row.sum() if row.sum() > 0 else row
        node, r, n = 0, spread(p[b, 0]), 1
        path[b, 0] = 0
        j = 1
        while j < use:
            x = int(tok[b, j])
            if par[b, j] != node or not 0 <= x < V or r.sum() == 0 or not allowed()[x]:
                j += 1
                continue
            if q is None:
                d = np.zeros(V)
                d[x] = 1.0
            else:
                d = spread(q[b, node])
            if uu[b, j] * d[x] < r[x]:
                if states is not None:
                    s = int(nxt[s, x])
                node = j
                path[b, n] = j
                n += 1
                r = spread(p[b, j])
            else:
                rest = np.maximum(r - d, 0.0)
                if q is None:
                    rest = r.copy()
                    rest[x] = 0.0
                if rest.sum() > 0:
                    r = rest / rest.sum()
            j += 1
        kept[b] = n
        if r.sum() > 0:
            at = int((np.cumsum(r) <= uu[b, 0]).sum())
            token[b] = min(at, int(np.nonzero(r)[0][-1]))
            if states is not None:
                state[b] = nxt[s, token[b]]
    return path, kept, token, state


class Pool:
    """Pages as Python lists."""

    def __init__(self, pages):
        self.table = pages.table.cpu().tolist()
        self.held = pages.held.cpu().tolist()
        self.stack = pages.free.cpu().tolist()[:int(pages.n_free)]
        self.n, self.size, self.per = pages.free.shape[0], pages.page_size, pages.table.shape[1]

    def resize(self, want):
        need = [-(-max(w, 0) // self.size) for w in want]
        back = []
        for b, n in enumerate(need):
            back += self.table[b][n:self.held[b]]
            for i in range(n, self.held[b]):
                self.table[b][i] = -1
            self.held[b] = min(self.held[b], n)
        self.stack += back[::-1]
        status, short = [], False
        for b, n in enumerate(need):
            if n > self.per:
                status.append(2)
            elif n > self.held[b] and (short or n - self.held[b] > len(self.stack)):
                short = True
                status.append(1)
            else:
                while self.held[b] < n:
                    self.table[b][self.held[b]] = self.stack.pop()
                    self.held[b] += 1
                status.append(0)
        return status

    def same(self, pages):
        assert pages.table.cpu().tolist() == self.table
        assert pages.held.cpu().tolist() == self.held
        assert int(pages.n_free) == len(self.stack)
        assert pages.free.cpu().tolist() == self.stack + [-1] * (self.n - len(self.stack))


def slot_map(table, n_pages, size, start, count, N):
    slot, seq, pos, offset = [], [], [], [0]
    for b, (s, c) in enumerate(zip(start, count)):
        for t in range(s, s + max(c, 0)):
            page = table[b][t // size] if 0 <= t // size < len(table[b]) else -1
            slot.append(page * size + t % size if 0 <= page < n_pages else -1)
            seq.append(b)
            pos.append(t)
        offset.append(min(len(slot), N))
    fill = [-1] * max(0, N - len(slot))
    return [(x + fill)[:N] for x in (slot, seq, pos)] + [offset]


def rotated(key, positions, base=10000.0, interleaved=False, mscale=1.0):
    """key [N, R] in 64 bits, rotated at positions [N]."""
    x = key.double().cpu().numpy()
    pos = positions.cpu().double().numpy()
    R = x.shape[1]
    y = x.copy()
    for i in range(R // 2):
        a = pos * base ** (-2.0 * i / R)
        p, q = (2 * i, 2 * i + 1) if interleaved else (i, i + R // 2)
        y[:, p] = mscale * (x[:, p] * np.cos(a) - x[:, q] * np.sin(a))
        y[:, q] = mscale * (x[:, p] * np.sin(a) + x[:, q] * np.cos(a))
    return y


def seen(mask, b, i, use):
    """Which drafted tokens token i of sequence b sees (mask words, or None: all)."""
    if mask is None:
        return [True] * use
    return [bool(int(mask[b, i, j // 64]) >> (j % 64) & 1) for j in range(use)]


def latent_attention(q, rows, latent, table, length, scale, mask=None, count=None):
    """(out, lse, sum_t p |c|, max_t scale sum_d |q_d c_d|): the last two scale the error.  A sequence and a drafted
    token at a time, on the rows that are seen alone."""
    B, T, H, D = q.shape
    n_pages, size = rows.shape[:2]
    out, weight = (torch.zeros(B, T, H, latent, dtype=torch.float64, device=q.device) for _ in range(2))
    lse = torch.full((B, T, H), -math.inf, dtype=torch.float64, device=q.device)
    top = torch.zeros(B, T, H, dtype=torch.float64, device=q.device)
    words = None if mask is None else mask.cpu()
    tab = table.cpu().long()
    for b in range(B):
        n = min(max(int(length[b]), 0), tab.shape[1] * size)
        use = T if count is None else min(max(int(count[b]), 0), T)
        end = min(n + use, tab.shape[1] * size)
        t = torch.arange(end)
        page = tab[b][t // size]
        there = (page >= 0) & (page < n_pages)
        at = (torch.where(there, page, 0) * size + t % size).to(q.device)
        for i in range(use):
            ok = there.clone()
            ok[n:] &= torch.tensor(seen(words, b, i, use)[:end - n], dtype=torch.bool)
            sel = at[ok.to(q.device)]
            if len(sel) == 0:
                continue
            c = rows.view(-1, D)[sel].double()
            s = scale * q[b, i].double() @ c.T
            p = torch.softmax(s, -1)
            out[b, i], weight[b, i] = p @ c[:, :latent], p @ c[:, :latent].abs()
            lse[b, i] = torch.logsumexp(s, -1)
            top[b, i] = (scale * q[b, i].double().abs() @ c.abs().T).amax(-1)
    return out, lse, weight, top
