"""Plain 64-bit implementations of the model-side operators, on the CPU, one element or one
row at a time where that is the clearest.  They share nothing with the package."""
from __future__ import annotations

import math

import numpy as np
import torch

# half a unit in the last place, relative to the value: the rounding of a stored result
HALF_ULP = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 2.0 ** -149, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}


def rope(x, positions, rot, base=10000.0, divide=1.0, interleaved=False, mscale=1.0, inverse=False):
    """x [N, H, D]: the first rot elements rotated by position * base^(-2i / rot) / divide."""
    x = x.detach().cpu().double().numpy()
    pos = positions.cpu().double().numpy()
    y = x.copy()
    for i in range(rot // 2):
        a = pos * (base ** (-2.0 * i / rot) / divide)
        if inverse:
            a = -a
        p, q = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
        c, s = np.cos(a)[:, None], np.sin(a)[:, None]
        y[:, :, p] = mscale * (x[:, :, p] * c - x[:, :, q] * s)
        y[:, :, q] = mscale * (x[:, :, p] * s + x[:, :, q] * c)
    return y


def pair_sum(x, rot, interleaved):
    """|x0| + |x1| of each element's pair (0 where nothing is rotated): scales the fp32 error."""
    a = np.abs(x.detach().cpu().double().numpy())
    s = np.zeros_like(a)
    for i in range(rot // 2):
        p, q = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
        s[:, :, p] = s[:, :, q] = a[:, :, p] + a[:, :, q]
    return s


def cached_rows(cache, page_table, b, n):
    """Slots 0 .. n - 1 of a sequence: keys and values [n, heads, dim] in 64 bits (NaN where no
    page holds the slot)."""
    pages, heads, size, dim = cache.k.shape
    out = []
    for x, scale in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
        full = x.float().cpu().double()
        if scale is not None:
            full = full * scale.cpu().double()[..., None]
        got = torch.full((n, heads, dim), math.nan, dtype=torch.float64)
        for t in range(n):
            if t // size >= page_table.shape[1]:
                continue
            page = int(page_table[b, t // size])
            if 0 <= page < pages:
                got[t] = full[page, :, t % size]
        out.append(got)
    return out


def held(cache, page_table, b, n):
    size = cache.k.shape[2]
    return [t // size < page_table.shape[1] and 0 <= int(page_table[b, t // size]) < cache.k.shape[0] for t in range(n)]


def attention(q, cache, page_table, length, mask=None, count=None, scale=None):
    """(out, lse, sum_t p |v|, max_t scale sum_d |q_d k_d|): the last two scale the error."""
    B, T, H, D = q.shape
    G = H // cache.k.shape[1]
    scale = D ** -0.5 if scale is None else scale
    out, weight = np.zeros((B, T, H, D)), np.zeros((B, T, H, D))
    lse, size = np.full((B, T, H), -np.inf), np.zeros((B, T, H))
    qd = q.detach().cpu().double()
    table = page_table.cpu()
    for b in range(B):
        n = int(length[b])
        use = T if count is None else int(count[b])
        k, v = cached_rows(cache, table, b, n + use)
        there = held(cache, table, b, n + use)
        for i in range(use):
            sees = []
            for t in range(n + use):
                j = t - n
                word = None if mask is None or j < 0 else int(mask[b, i, j // 64])
                if there[t] and (j < 0 or mask is None or word >> (j % 64) & 1):
                    sees.append(t)
            if not sees:
                continue
            for h in range(H):
                kk, vv = k[sees, h // G], v[sees, h // G]
                s = scale * (kk @ qd[b, i, h])
                lse[b, i, h] = torch.logsumexp(s, 0)
                p = torch.softmax(s, 0)
                out[b, i, h] = p @ vv
                weight[b, i, h] = p @ vv.abs()
                size[b, i, h] = (kk.abs() @ qd[b, i, h].abs()).max() * abs(scale)
    return out, lse, weight, size


def tree_seen(parents):
    """seen[j]: the set of tokens that token j of one tree sees."""
    seen = []
    for j, p in enumerate(parents):
        seen.append((seen[p] if 0 <= p < j else set()) | {j})
    return seen


def beam(logp, scores, top, states=None, next_state=None):
    """The best cells by one fp32 addition each, sorted by (-value, index)."""
    N, K, V = logp.shape
    x = logp.float().cpu().numpy()
    s = scores.cpu().numpy()
    score = np.full((N, top), -np.inf, np.float32)
    parent, token, state = (np.full((N, top), -1, np.int32) for _ in range(3))
    for n in range(N):
        with np.errstate(invalid="ignore"):
            v = s[n][:, None] + x[n]
        ok = v > -np.inf
        for k in range(K):
            if not s[n, k] > -np.inf:
                ok[k] = False
            elif states is not None:
                st = int(states[n, k])
                ok[k] &= (next_state[st] >= 0) if 0 <= st < next_state.shape[0] else False
        flat = np.nonzero(ok.ravel())[0]
        order = flat[np.lexsort((flat, -v.ravel()[flat].astype(np.float64)))][:top]
        for i, c in enumerate(order):
            score[n, i], parent[n, i], token[n, i] = v.ravel()[c], c // V, c % V
            if states is not None:
                state[n, i] = next_state[int(states[n, c // V]), c % V]
    return score, parent, token, state
