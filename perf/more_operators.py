"""Operators of a program that drafts, verifies and serves over a latent cache, as measured cases.

Four operators that belong together: pages handed out and slots mapped on the device, a paged cache
of one latent vector a token with its writes, attention of drafted tokens over it, and the
verification of drafted tokens against the target's probabilities.

`own` chooses between the plain form (elementary torch operations) and the calls of the package.
Every case is a dict of plain values; `prepare` makes its inputs on the GPU from a seed, `run` is
one pass and `exact` the same outputs from the definitions in 64 bits.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
ES = {"bf16": 2, "fp16": 2, "fp32": 4}
ACCEPTED = 2.0 / 3.0  # the share of drafted tokens that the verification inputs' distributions accept


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # a chain of four sampled tokens of one sequence: latency
        dict(name="verify_step", op="verify", batch=1, beams=1, depth=4, vocab=32000, draft=True, states=0, dtype="fp32"),
        # a serving batch's chains of eight sampled tokens over a large vocabulary
        dict(name="verify_batch", op="verify", batch=64, beams=1, depth=8, vocab=151936, draft=True, states=0,
             dtype="fp32"),
        # trees of four beams under a DFA of 512 states: the beams are chosen, not sampled
        dict(name="verify_tree", op="verify", batch=16, beams=4, depth=4, vocab=151936, draft=False, states=512,
             dtype="bf16"),
        # one decoding step of 64 sequences: room for a draft of 8, its slots, what was not accepted given back
        dict(name="pages_step", op="pages", batch=64, page=16, ctx=4096, tokens=8, turnover=False),
        # 256 sequences of which half end while the other half's prompts arrive, and back
        dict(name="pages_turnover", op="pages", batch=256, page=16, ctx=8192, tokens=256, turnover=True),
        # a draft of 5 written for each of 64 sequences, and its accepted path moved together
        dict(name="latent_write_draft", op="write", batch=64, tokens=5, latent=512, rope=64, dtype="bf16", page=64,
             ctx=512, keep=True),
        # prompts of 16 sequences, 32768 tokens in all
        dict(name="latent_write_prompt", op="write", batch=16, tokens=2048, latent=512, rope=64, dtype="bf16", page=64,
             ctx=0, keep=False),
        # a small batch's next token over a short context: latency
        dict(name="latent_step", op="attend", batch=4, tokens=1, heads=16, latent=512, rope=64, dtype="bf16", page=16,
             ctx=509, mask="chain", ragged=True),
        # a serving batch's next tokens over ragged contexts
        dict(name="latent_batch", op="attend", batch=32, tokens=1, heads=32, latent=512, rope=64, dtype="bf16", page=64,
             ctx=8192, mask="chain", ragged=True),
        # the same with many heads: two blocks of rows read each slot
        dict(name="latent_heads", op="attend", batch=16, tokens=1, heads=128, latent=512, rope=64, dtype="bf16", page=64,
             ctx=8192, mask="chain", ragged=False),
        # a tree of 16 drafted tokens over two very long contexts, smaller latents
        dict(name="latent_tree_long", op="attend", batch=2, tokens=16, heads=16, latent=256, rope=32, dtype="fp16",
             page=32, ctx=98304, mask="tree", ragged=False),
        # a block of 32 masked positions that see one another, over the decoded prefix
        dict(name="latent_block", op="attend", batch=16, tokens=32, heads=32, latent=512, rope=64, dtype="bf16", page=64,
             ctx=4096, mask="block", ragged=False),
    ]


def _spread(rng, lo, hi):
    """An integer between lo and hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _cost(case):
    w = work(case)
    return w["bytes"] / 6.7e12 + w["flops"] / 1.9e15


def draw(rng):
    """One more case of the ranges above: its operator first, then sizes over the whole range."""
    op = rng.choice(["verify", "verify", "pages", "write", "attend", "attend"])
    most = max(_cost(c) for c in listed() if c["op"] == op)
    while True:
        page = rng.choice([8, 16, 32, 64, 128])
        latent, rope = rng.choice([128, 256, 384, 512, 512]), rng.choice([16, 32, 64, 64])
        dtype = rng.choice(["bf16", "fp16"])
        if op == "verify":
            c = dict(op=op, batch=_spread(rng, 1, 64), beams=rng.choice([1, 1, 2, 4]), depth=rng.randint(1, 8),
                     vocab=_spread(rng, 100, 151936), draft=rng.random() < 0.6, states=rng.choice([0, 0, 5, 64, 512]),
                     dtype=rng.choice(["fp32", "fp32", "bf16", "fp16"]))
        elif op == "pages":
            c = dict(op=op, batch=_spread(rng, 1, 1024), page=page, ctx=_spread(rng, 1, 16384), tokens=_spread(rng, 1, 256),
                     turnover=rng.random() < 0.5)
        elif op == "write":
            c = dict(op=op, batch=_spread(rng, 1, 64), tokens=_spread(rng, 1, 2048), latent=latent, rope=rope, dtype=dtype,
                     page=page, ctx=_spread(rng, 1, 2048) - 1, keep=rng.random() < 0.5)
            c["keep"] = c["keep"] and c["tokens"] <= 64
        else:
            c = dict(op=op, batch=_spread(rng, 1, 32), tokens=rng.choice([1, 1, _spread(rng, 2, 64)]),
                     heads=rng.choice([1, 3, 8, 16, 32, 40, 128]), latent=latent, rope=rope, dtype=dtype, page=page,
                     ctx=_spread(rng, 1, 98304), mask=rng.choice(["chain", "tree", "block"]), ragged=rng.random() < 0.5)
        scores = c["batch"] * c["tokens"] * c["heads"] * (c["ctx"] + c["tokens"]) if op == "attend" else 0
        if _cost(c) <= most and scores <= 1 << 28:  # what the plain form holds at once
            return c


def _lengths(c):
    """The cached length of each sequence: all `ctx`, or ragged down to an empty one."""
    B, n = c["batch"], c["ctx"]
    if not c.get("ragged", True):
        return [n] * B
    out = [max(0, n * (B - b) // B - (5 * b) % 7) for b in range(B)]
    if B > 3:
        out[-1] = 0
    return out


def _drafted(c):
    """How many new tokens of each sequence are in use."""
    T = c["tokens"]
    return [max(1, T - b % 3) if c.get("ragged", True) else T for b in range(c["batch"])]


def _wanted(c):
    """Slots wanted of a pool: (before the pass and after it, in the middle of it)."""
    n, T = _lengths(c), _drafted(c)
    if c["turnover"]:
        return ([x if b % 2 else 0 for b, x in enumerate(n)], [0 if b % 2 else x + T[b] for b, x in enumerate(n)])
    return [x + max(1, T[b] * (b % 4) // 4) for b, x in enumerate(n)], [x + T[b] for b, x in enumerate(n)]


def work(case):
    """Bytes and operations that one pass cannot do without."""
    c = case
    if c["op"] == "verify":
        # the rows of the nodes that are visited; beams below the first token agree less often
        below = sum((ACCEPTED if c["draft"] else 0.4) ** k for k in range(c["depth"]))
        cells = c["batch"] * (1 + ACCEPTED * below) * c["vocab"]
        both = 2 if c["draft"] else 1
        return {"bytes": cells * (both * ES[c["dtype"]] + (0.125 if c["states"] else 0)), "flops": both * cells}
    if c["op"] == "pages":
        a, b = ([-(-x // c["page"]) for x in w] for w in _wanted(c))
        moved = 2.0 * sum(abs(x - y) for x, y in zip(a, b))
        tokens = float(sum(_drafted(c)))
        return {"bytes": 8 * moved + 12 * tokens + 32.0 * c["batch"], "flops": 4 * (moved + tokens + c["batch"])}
    dim = c["latent"] + c["rope"]
    if c["op"] == "write":
        n = float(sum(_drafted(c)))
        kept = sum((t + 1) // 2 for t in _drafted(c)) if c["keep"] else 0
        return {"bytes": 2.0 * ES[c["dtype"]] * dim * (n + kept), "flops": 3.0 * n * c["rope"]}
    keys = [n + t for n, t in zip(_lengths(c), _drafted(c))]
    rows = float(c["batch"] * c["tokens"] * c["heads"])
    pairs = c["heads"] * sum(k * t for k, t in zip(keys, _drafted(c)))
    return {"bytes": float(ES[c["dtype"]]) * (sum(keys) * dim + rows * (dim + c["latent"])) + 4 * rows,
            "flops": 2.0 * (dim + c["latent"]) * pairs}


# ------------------------------------------------------------------ inputs

def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _phases(rot):
    """The angle of each rotated pair per position, in turns as a 64-bit fixed-point fraction (an
    int64 holding the bits)."""
    got = []
    for i in range(rot // 2):
        bits = int(10000.0 ** (-2.0 * i / rot) / (2 * math.pi) * 2.0 ** 64) % (1 << 64)
        got.append(bits - (1 << 64) if bits >= 1 << 63 else bits)
    return torch.tensor(got, dtype=torch.int64, device="cuda")


def _pages(c, gen, slots):
    """A page table over a pool with a few pages to spare, in no order."""
    per = max(1, -(-slots // c["page"]))
    n = c["batch"] * per + 3
    order = torch.randperm(n, generator=gen, device="cuda")[:c["batch"] * per]
    return n, order.to(torch.int32).view(c["batch"], per)


def _tree_words(c, seed):
    """Which drafted tokens each drafted token sees, as 64-bit words: None = all of them."""
    B, T = c["batch"], c["tokens"]
    if c["mask"] == "block":
        return None
    import random
    rng = random.Random(seed)
    rows = []
    for _ in range(B):
        seen = []
        for j in range(T):
            parent = j - 1 if c["mask"] == "chain" else rng.randint(-1, j - 1) if j else -1
            seen.append((seen[parent] if parent >= 0 else 0) | 1 << j)
        rows.append([[_signed(s >> 64 * w & (1 << 64) - 1) for w in range(-(-T // 64))] for s in seen])
    return torch.tensor(rows, dtype=torch.int64, device="cuda")


def _signed(word):
    return word - (1 << 64) if word >= 1 << 63 else word


def _parents(c):
    """The pending token, then the beams, one after another."""
    n = 1 + c["beams"] * c["depth"]
    return [-1] + [0 if (j - 1) % c["depth"] == 0 else j - 1 for j in range(1, n)]


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)

    s = {"case": c}
    if c["op"] == "verify":
        _prepare_verify(s, c, gen, normal)
    elif c["op"] == "pages":
        B, G = c["batch"], c["page"]
        before, during = _wanted(c)
        per = -(-(c["ctx"] + c["tokens"]) // G)
        s["n_pages"] = 5 + max(sum(-(-x // G) for x in w) for w in (before, during))
        held = [-(-x // G) for x in before]
        order = torch.randperm(s["n_pages"], generator=gen, device="cuda").int()
        table = torch.full((B, per), -1, dtype=torch.int32, device="cuda")
        use = torch.arange(per, device="cuda") < _ints(held)[:, None]
        table[use] = order[:sum(held)]
        free = torch.full((s["n_pages"],), -1, dtype=torch.int32, device="cuda")
        free[:s["n_pages"] - sum(held)] = order[sum(held):]
        s.update(table=table, free=free, held=_ints(held), n_free=_ints([s["n_pages"] - sum(held)]),
                 before=_ints(before), during=_ints(during), tokens=B * c["tokens"])
        drafted = [min(t, w) for t, w in zip(_drafted(c), during)]
        s["start"] = _ints([w - t for t, w in zip(drafted, during)])
        s["count"] = _ints(drafted)
    elif c["op"] == "write":
        B, T, dt = c["batch"], c["tokens"], DT[c["dtype"]]
        n, s["table"] = _pages(c, gen, c["ctx"] + T)
        dim = c["latent"] + c["rope"]
        s["rows"] = normal(n, c["page"], dim).to(dt)
        start, count = _lengths(c), _drafted(c)
        total = sum(count)
        down = normal(total, dim).to(dt)  # as the down projection leaves them
        s["latent"], s["key"] = down[:, :c["latent"]], down[:, c["latent"]:]
        s["length"] = _ints(start)
        seq = torch.repeat_interleave(torch.arange(B, device="cuda"), _ints(count).long())
        first = torch.cumsum(_ints(count), 0) - _ints(count)
        s["pos"] = (s["length"][seq] + torch.arange(total, device="cuda") - first[seq]).int()
        s["slot"] = (s["table"][seq, (s["pos"] // c["page"]).long()] * c["page"] + s["pos"] % c["page"]).int()
        s["phase"] = _phases(c["rope"])
        if c["keep"]:  # every other drafted token is on the accepted path
            path = torch.full((B, T), -1, dtype=torch.int32, device="cuda")
            for b, t in enumerate(count):
                path[b, :(t + 1) // 2] = torch.arange(0, t, 2, device="cuda")
            s["path"] = path
    else:
        B, T, H, dt = c["batch"], c["tokens"], c["heads"], DT[c["dtype"]]
        dim = c["latent"] + c["rope"]
        n, s["table"] = _pages(c, gen, c["ctx"] + T)
        s["q"] = normal(B, T, H, dim).to(dt)
        s["rows"] = normal(n, c["page"], dim).to(dt)
        s["length"], s["count"] = _ints(_lengths(c)), _ints(_drafted(c))
        s["mask"] = _tree_words(c, seed)
        s["scale"] = (128 + c["rope"]) ** -0.5  # of the expanded keys: 128 elements of their own and the rotary ones
        if own:  # the workspace and the outputs that a program keeps from step to step
            from constrained_decoding_diffusion_gb300 import lm
            s["attend"] = lm.LatentAttention(B, T, H, c["latent"], c["rope"], dt)
    return s


def _prepare_verify(s, c, gen, normal):
    B, V, S, dt = c["batch"], c["vocab"], c["states"], DT[c["dtype"]]
    parents = _parents(c)
    T = len(parents)
    guess = normal(B, T, V)
    s["target"] = torch.softmax(6 * (math.sqrt(0.96) * guess + 0.2 * normal(B, T, V)), -1).to(dt)
    guess *= 6
    s["draft"] = torch.softmax(guess, -1).to(dt) if c["draft"] else None
    s["parents"] = _ints([parents] * B)
    s["u"] = torch.rand((B, T), generator=gen, device="cuda")
    s["state"] = s["next"] = s["live"] = None
    if S:
        to = torch.randint(0, S, (S, V), generator=gen, device="cuda", dtype=torch.int16)
        dead = torch.rand((S, V), generator=gen, device="cuda") < 0.7
        s["next"] = to.masked_fill_(dead, -1)
        bits = torch.zeros((S, -(-V // 32) * 32), dtype=torch.int32, device="cuda")
        bits[:, :V] = (s["next"] >= 0).to(torch.int32)
        place = torch.arange(32, device="cuda", dtype=torch.int32)
        s["live"] = torch.bitwise_left_shift(bits.view(S, -1, 32), place).sum(-1, dtype=torch.int32)
        s["state"] = torch.randint(0, S, (B,), generator=gen, device="cuda", dtype=torch.int32)
    # the draft, node by node: sampled from the guess, or the best that are left
    tokens = torch.zeros((B, T), dtype=torch.int32, device="cuda")
    tokens[:, 0] = torch.randint(0, V, (B,), generator=gen, device="cuda", dtype=torch.int32)
    state = [s["state"]] + [None] * (T - 1)
    for j in range(1, T):
        p = parents[j]
        x = guess[:, p]
        if S:
            x = x.masked_fill(s["next"][state[p].long()] < 0, -math.inf)
        if c["draft"]:
            tokens[:, j] = (x - torch.log(-torch.log(torch.rand((B, V), generator=gen, device="cuda")))).argmax(-1)
        else:
            tokens[:, j] = torch.topk(x, c["beams"]).indices[:, (j - 1) // c["depth"] if p == 0 else 0]
        if S:
            state[j] = s["next"][state[p].long(), tokens[:, j].long()].int().clamp(min=0)
    s["tokens"] = tokens
    if own:
        from constrained_decoding_diffusion_gb300 import lm
        s["verify"] = lm.Verify(B, T, V, dt)


# ------------------------------------------------------------------ one pass

def run(state):
    return (_own if own else _plain)[state["case"]["op"]](state, state["case"])


# -- the plain forms

def _plain_verify(s, c):
    """Nodes in index order: a child of the current node is accepted or leaves the distribution that is left.
    In 64 bits: a draw is a comparison with a sum over the vocabulary."""
    B, T, V = s["target"].shape
    every = torch.arange(B, device="cuda")
    cur = torch.zeros(B, dtype=torch.long, device="cuda")
    state = s["state"].long() if c["states"] else None
    path = torch.full((B, T), -1, dtype=torch.int32, device="cuda")
    path[:, 0] = 0
    kept = torch.ones(B, dtype=torch.long, device="cuda")

    def rows(x):
        x = x[every, cur].double()
        return torch.where(s["next"][state] >= 0, x, 0.0) if c["states"] else x

    p = rows(s["target"])
    q = rows(s["draft"]) if c["draft"] else None
    left, lam = p, torch.zeros(B, dtype=torch.float64, device="cuda")
    total = left.sum(-1)
    for j in range(1, T):
        x = s["tokens"][:, j].long()
        test = s["parents"][:, j].long() == cur
        u = s["u"][:, j].double()
        mine = left[every, x]
        if c["draft"]:
            all_q = q.sum(-1)
            take = test & (u * total * q[every, x] < mine * all_q)
            lam_next = lam + total / torch.where(all_q > 0, all_q, 1.0)
            less = (p - lam_next[:, None] * q).clamp(min=0)
        else:
            take = test & (u * total < mine)
            lam_next = lam
            less = left.clone()
            less[every, x] = 0.0
        rest = less.sum(-1)
        drop = test & ~take & (rest > 0)
        left = torch.where(drop[:, None], less, left)
        lam = torch.where(drop, lam_next, lam)
        cur = torch.where(take, j, cur)
        if c["states"]:
            state = torch.where(take, s["next"][state, x].long(), state)
        path[every, kept.clamp(max=T - 1)] = torch.where(take, j, path[every, kept.clamp(max=T - 1)]).int()
        kept = kept + take
        p = torch.where(take[:, None], rows(s["target"]), p)
        if c["draft"]:
            q = torch.where(take[:, None], rows(s["draft"]), q)
        left = torch.where(take[:, None], p, left)
        lam = torch.where(take, 0.0, lam)
        total = left.sum(-1)
    below = (torch.cumsum(left, -1) <= (s["u"][:, 0].double() * total)[:, None]).sum(-1)
    last = V - 1 - (left > 0).flip(-1).int().argmax(-1)
    token = torch.where(total > 0, torch.minimum(below, last), -1)
    got = {"path": path, "kept": kept.int(), "token": token.int()}
    if c["states"]:
        got["state"] = torch.where(token >= 0, s["next"][state, token.clamp(min=0)].long(), -1).int()
    return got


def _plain_resize(s, c, want):
    """Pages past what is wanted go back to the pool, the first on top; then sequences take theirs from the
    top, in order, while there are enough."""
    B, per = s["table"].shape
    at = torch.arange(per, device="cuda")
    held = s["held"].long()
    need = (want.long().clamp(min=0) + c["page"] - 1) // c["page"]
    back = (at >= need[:, None]) & (at < held[:, None])
    n_free = s["n_free"].long()
    grow = torch.where(need <= per, (need - held).clamp(min=0), 0)
    returned = back.sum()
    there = n_free + returned
    granted = (torch.cumsum(grow, 0) <= there) | (grow == 0)
    status = torch.where(need > per, 2, torch.where(granted, 0, 1)).int()
    free = torch.cat([s["free"], s["free"].new_zeros(1)])  # the last place takes what goes nowhere
    rank = torch.cumsum(back.flatten(), 0).view(B, per) - 1
    free[torch.where(back, there - 1 - rank, s["n_pages"])] = s["table"]
    take = (at >= held[:, None]) & (at < need[:, None]) & (granted & (need <= per))[:, None]
    rank = torch.cumsum(take.flatten(), 0).view(B, per) - 1
    new = free[torch.where(take, there - 1 - rank, s["n_pages"])]
    s["table"].copy_(torch.where(back, -1, torch.where(take, new, s["table"])))
    s["free"].copy_(free[:-1])
    s["n_free"].copy_(there - take.sum())
    s["held"].copy_(torch.where(need <= per, torch.where(granted, need, held), held))
    return status


def _plain_pages(s, c):
    got = {"status": _plain_resize(s, c, s["during"])}
    offset = torch.nn.functional.pad(torch.cumsum(s["count"], 0), (1, 0))
    n = torch.arange(s["tokens"], device="cuda")
    seq = torch.searchsorted(offset, n, right=True) - 1
    use = n < offset[-1]
    seq = seq.clamp(max=c["batch"] - 1)
    pos = s["start"][seq] + n - offset[seq]
    page = s["table"][seq, (pos // c["page"]).clamp(0, s["table"].shape[1] - 1)]
    slot = torch.where(page >= 0, page * c["page"] + pos % c["page"], -1)
    for name, x in (("slot", slot), ("seq", seq), ("pos", pos)):
        got[name] = torch.where(use, x, -1).int()
    got["offset"] = offset.int()
    got["status_after"] = _plain_resize(s, c, s["before"])
    there = torch.arange(s["n_pages"], device="cuda") < s["n_free"]
    got.update(table=s["table"], held=s["held"], n_free=s["n_free"], free=torch.where(there, s["free"], -1))
    return got


def _plain_write(s, c):
    half = c["rope"] // 2
    turns = s["pos"].long()[:, None] * s["phase"]  # wraps around: whole turns drop out
    angle = (turns >> 32).float() * (2 * math.pi / 2 ** 32)
    cos, sin = torch.cos(angle), torch.sin(angle)
    x = s["key"].float()
    a, b = x[:, :half], x[:, half:]
    row = torch.cat([s["latent"].float(), a * cos - b * sin, a * sin + b * cos], -1).to(s["rows"].dtype)
    flat = s["rows"].view(-1, row.shape[1])
    flat[s["slot"].long()] = row
    if c["keep"]:
        use = s["path"] >= 0
        i = torch.arange(c["tokens"], device="cuda")

        def places(slot):
            page = torch.gather(s["table"].long(), 1, (slot // c["page"]).clamp(max=s["table"].shape[1] - 1))
            return page * c["page"] + slot % c["page"]
        src = places(s["length"].long()[:, None] + s["path"].long().clamp(min=0))
        dst = places(s["length"].long()[:, None] + i)
        flat[dst[use]] = flat[src[use]]
    return s["rows"]


def _plain_attend(s, c):
    B, T, H, L = c["batch"], c["tokens"], c["heads"], c["latent"]
    rows = s["rows"][s["table"].long()].float().flatten(1, 2)  # [batch, slots, latent + rope]
    n, use = s["length"][:, None, None], s["count"][:, None, None]
    at = torch.arange(rows.shape[1], device="cuda")
    j = (at - n).clamp(0, T - 1).expand(B, T, -1)
    tree = torch.ones((B, T, T), dtype=torch.bool, device="cuda")
    if s["mask"] is not None:
        place = torch.arange(T, device="cuda")
        tree = (s["mask"][:, :, place // 64] >> (place % 64)) & 1 != 0
    sees = (at < n) | ((at < n + use) & torch.gather(tree, 2, j))
    sees = (sees & (torch.arange(T, device="cuda")[:, None] < use)).repeat_interleave(H, 1)
    x = torch.matmul(s["q"].float().view(B, T * H, -1), rows.transpose(1, 2)) * s["scale"]
    x = torch.where(sees, x, -math.inf)
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(top > -math.inf, top, 0.0))
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p, rows[..., :L]) / torch.where(total > 0, total, 1.0)
    lse = (top + torch.log(total)).squeeze(-1)
    return {"out": out.view(B, T, H, L).to(s["q"].dtype), "lse": lse.view(B, T, H)}


_plain = {"verify": _plain_verify, "pages": _plain_pages, "write": _plain_write, "attend": _plain_attend}


# -- the package's calls

def _own_verify(s, c):
    path, kept, token, state = s["verify"](s["target"], s["tokens"], s["parents"], s["u"], draft=s["draft"],
                                           states=s["state"], next=s["next"], live=s["live"])
    got = {"path": path, "kept": kept, "token": token}
    if c["states"]:
        got["state"] = state
    return got


def _own_pages(s, c):
    from constrained_decoding_diffusion_gb300 import lm
    pages = lm.PageTables(s["table"], s["held"], s["free"], s["n_free"], c["page"])
    got = {"status": lm.fa_pages_resize(pages, s["during"])}
    got["slot"], got["seq"], got["pos"], got["offset"] = lm.fa_slot_map(pages, s["start"], s["count"], s["tokens"])
    got["status_after"] = lm.fa_pages_resize(pages, s["before"])
    got.update(table=s["table"], held=s["held"], n_free=s["n_free"], free=s["free"])
    return got


def _own_write(s, c):
    from constrained_decoding_diffusion_gb300 import lm
    cache = lm.LatentCache(s["rows"], c["latent"])
    lm.fa_latent_write(cache, s["latent"], s["key"], s["slot"], positions=s["pos"], phase=s["phase"])
    if c["keep"]:
        lm.fa_latent_keep(cache, s["table"], s["length"], s["path"])
    return s["rows"]


def _own_attend(s, c):
    from constrained_decoding_diffusion_gb300 import lm
    out, lse = s["attend"](s["q"], lm.LatentCache(s["rows"], c["latent"]), s["table"], s["length"], scale=s["scale"],
                           mask=s["mask"], count=s["count"])
    return {"out": out, "lse": lse}


_own = {"verify": _own_verify, "pages": _own_pages, "write": _own_write, "attend": _own_attend}


# ------------------------------------------------------------------ the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"verify": _exact_verify, "pages": _exact_pages, "write": _exact_write, "attend": _exact_attend}[case["op"]](s, case)


def _exact_verify(s, c):
    """A sequence at a time, with the distributions themselves: r is what is left of the target's."""
    B, T, V = s["target"].shape
    parents = _parents(c)
    got = {"path": [], "kept": [], "token": [], "state": []}
    u, tokens = s["u"].double().cpu().tolist(), s["tokens"].cpu().tolist()
    for b in range(B):
        state = int(s["state"][b]) if c["states"] else 0

        def spread(x, j):
            x = x[b, j].double()
            if c["states"]:
                x = x * (s["next"][state] >= 0)
            return x / x.sum()
        path, open_children = [0], [j for j in range(T) if parents[j] == 0]
        r = spread(s["target"], 0)
        while open_children:
            j = open_children.pop(0)
            x = tokens[b][j]
            if c["draft"]:
                q = spread(s["draft"], path[-1])
            else:
                q = torch.zeros(V, dtype=torch.float64, device="cuda")
                q[x] = 1.0
            if bool(u[b][j] * q[x] < r[x]):
                path.append(j)
                if c["states"]:
                    state = int(s["next"][state, x])
                r = spread(s["target"], j)
                open_children = [i for i in range(T) if parents[i] == j]
            else:
                rest = (r - q).clamp(min=0)
                if not c["draft"]:
                    rest = r.clone()
                    rest[x] = 0.0
                if bool(rest.sum() > 0):
                    r = rest / rest.sum()
        token = int((torch.cumsum(r, 0) <= u[b][0]).sum())
        token = min(token, int(r.nonzero()[-1]))
        got["path"].append(path + [-1] * (T - len(path)))
        got["kept"].append(len(path))
        got["token"].append(token)
        if c["states"]:
            got["state"].append(int(s["next"][state, token]))
    if not c["states"]:
        del got["state"]
    return {k: _ints(v) for k, v in got.items()}


def _exact_pages(s, c):
    """With Python lists: a stack, and one sequence after another."""
    table, held = s["table"].cpu().tolist(), s["held"].cpu().tolist()
    stack = s["free"].cpu().tolist()[:int(s["n_free"])]
    got = {}

    def resize(want):
        want = want.cpu().tolist()
        back, status = [], []
        for b, w in enumerate(want):
            need = -(-max(w, 0) // c["page"])
            back += table[b][need:held[b]]
            for i in range(need, held[b]):
                table[b][i] = -1
            held[b] = min(held[b], need)
        stack.extend(reversed(back))
        short = False
        for b, w in enumerate(want):
            need = -(-max(w, 0) // c["page"])
            if need > len(table[b]):
                status.append(2)
            elif need > held[b] and (short or need - held[b] > len(stack)):
                short = True
                status.append(1)
            else:
                for i in range(held[b], need):
                    table[b][i] = stack.pop()
                held[b] = need
                status.append(0)
        return _ints(status)

    got["status"] = resize(s["during"])
    slot, seq, pos, offset = [], [], [], [0]
    for b, (first, n) in enumerate(zip(s["start"].cpu().tolist(), s["count"].cpu().tolist())):
        for t in range(first, first + n):
            page = table[b][t // c["page"]]
            slot.append(page * c["page"] + t % c["page"] if page >= 0 else -1)
            seq.append(b)
            pos.append(t)
        offset.append(len(slot))
    for name, x in (("slot", slot), ("seq", seq), ("pos", pos)):
        got[name] = _ints(x + [-1] * (s["tokens"] - len(x)))
    got["offset"] = _ints(offset)
    got["status_after"] = resize(s["before"])
    got.update(table=_ints(table), held=_ints(held), n_free=_ints([len(stack)]),
               free=_ints(stack + [-1] * (s["n_pages"] - len(stack))))
    return got


def _exact_write(s, c):
    rows = s["rows"].double()
    flat = rows.view(-1, rows.shape[-1])
    new = torch.cat([s["latent"], s["key"]], -1).double()
    half, first = c["rope"] // 2, c["latent"]
    for i in range(half):
        turn = torch.polar(torch.ones(s["pos"].shape, dtype=torch.float64, device="cuda"),
                           s["pos"].double() * 10000.0 ** (-2.0 * i / c["rope"]))
        z = torch.complex(s["key"][:, i].double(), s["key"][:, i + half].double()) * turn
        new[:, first + i], new[:, first + half + i] = z.real, z.imag
    flat[s["slot"].long()] = new
    if c["keep"]:
        G = c["page"]
        table, path, length = s["table"].cpu().tolist(), s["path"].cpu().tolist(), s["length"].cpu().tolist()
        for b in range(c["batch"]):
            for i, j in enumerate(path[b]):
                if j >= 0:
                    src, dst = length[b] + j, length[b] + i
                    rows[table[b][dst // G], dst % G] = rows[table[b][src // G], src % G].clone()
    return rows


def _exact_attend(s, c):
    B, T, H, L, G = c["batch"], c["tokens"], c["heads"], c["latent"], c["page"]
    out = torch.zeros((B, T, H, L), dtype=torch.float64, device="cuda")
    lse = torch.full((B, T, H), -math.inf, dtype=torch.float64, device="cuda")
    words = None if s["mask"] is None else s["mask"].cpu().tolist()
    for b, (n, use) in enumerate(zip(_lengths(c), _drafted(c))):
        rows = s["rows"][s["table"][b, :-(-(n + use) // G)].long()].flatten(0, 1)[:n + use].double()
        sees = torch.ones((use, n + use), dtype=torch.bool)
        if words is not None:
            for i in range(use):
                for j in range(use):
                    sees[i, n + j] = bool(words[b][i][j // 64] >> (j % 64) & 1)
        x = torch.einsum("thd,nd->thn", s["q"][b, :use].double(), rows) * s["scale"]
        x = x.masked_fill(~sees.cuda()[:, None], -math.inf)
        lse[b, :use] = torch.logsumexp(x, -1)
        out[b, :use] = torch.einsum("thn,nd->thd", torch.softmax(x, -1), rows[:, :L])
    return {"out": out, "lse": lse}
