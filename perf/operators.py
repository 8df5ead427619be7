"""The language-model operators beside the constrained step, as measured cases.

Four operators that a program needs to run a denoiser or a drafter next to the automaton:
rotary positions, a paged key/value cache that is quantised as it is written, attention of a
block or a tree of drafted tokens over that cache, and beam selection under an automaton with
the reordering of the beams' histories.

`own` chooses between the plain form (elementary torch operations in 32 bits) and the calls of
the package.  Every case is a dict of plain values; `prepare` makes its inputs on the GPU from a
seed, `run` is one pass and `exact` the same outputs from the definitions in 64 bits.
"""
import math

import torch

own = False

E4M3_MAX = 448.0
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
ES = {"bf16": 2, "fp16": 2, "fp32": 4, "e4m3": 1}


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # one decoding step of a batch of 16: a query token of 32 heads each, far into a context
        dict(name="rope_step", op="rope", n=16, heads=32, dim=128, rot=128, interleaved=False, dtype="bf16",
             scaled=True, far=131072, grad=False),
        # a training batch of 16 sequences of 512 positions: half of each head rotated, and the
        # gradient's way back
        dict(name="rope_train", op="rope", n=8192, heads=32, dim=128, rot=64, interleaved=True, dtype="bf16",
             scaled=False, far=512, grad=True),
        # a single token appended to each of 16 ragged sequences, quantised to 8 bits
        dict(name="write_step", op="write", batch=16, tokens=1, kv_heads=8, dim=128, rot=128, interleaved=False,
             dtype="bf16", fmt="e4m3", page=64, ctx=4096, ragged=True),
        # a prompt of 2048 tokens written for 16 sequences
        dict(name="write_prompt", op="write", batch=16, tokens=2048, kv_heads=8, dim=128, rot=128, interleaved=False,
             dtype="bf16", fmt="e4m3", page=64, ctx=0, ragged=False),
        # a few short sequences read back from an unquantised cache: odd lengths, small pages
        dict(name="read_short", op="read", batch=3, kv_heads=4, dim=64, dtype="fp16", fmt="fp16", page=16, ctx=509,
             ragged=True),
        # a batch of long sequences read back in full
        dict(name="read_long", op="read", batch=16, kv_heads=8, dim=128, dtype="bf16", fmt="e4m3", page=64, ctx=8192,
             ragged=False),
        # a small batch's next token over a short context: latency
        dict(name="attend_step", op="attend", batch=4, tokens=1, kv_heads=8, group=4, dim=128, dtype="bf16",
             fmt="bf16", page=16, ctx=509, mask="chain", ragged=True),
        # a serving batch's next tokens over ragged contexts in an 8-bit cache
        dict(name="attend_batch", op="attend", batch=32, tokens=1, kv_heads=8, group=4, dim=128, dtype="bf16",
             fmt="e4m3", page=64, ctx=8192, mask="chain", ragged=True),
        # a tree of 16 drafted tokens verified over two very long contexts
        dict(name="attend_tree_long", op="attend", batch=2, tokens=16, kv_heads=8, group=4, dim=128, dtype="bf16",
             fmt="e4m3", page=64, ctx=98304, mask="tree", ragged=False),
        # a block of 64 masked positions that see one another, over the decoded prefix
        dict(name="attend_block", op="attend", batch=16, tokens=64, kv_heads=8, group=4, dim=128, dtype="bf16",
             fmt="bf16", page=64, ctx=8192, mask="block", ragged=False),
        # four beams over a vocabulary of 32000 under a DFA of 64 states
        dict(name="beam_small", op="beam", batch=1, beams=4, vocab=32000, top=4, states=64, dead=0.7, dtype="fp32",
             length=128),
        # 16 sequences of 16 beams over a vocabulary of 151936 under a DFA of 512 states
        dict(name="beam_large", op="beam", batch=16, beams=16, vocab=151936, top=16, states=512, dead=0.9,
             dtype="bf16", length=512),
    ]


def _spread(rng, lo, hi):
    """An integer between lo and hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """One more case of the ranges above: its operator first, then sizes over the whole range."""
    most = {}
    for c in listed():
        w = work(c)
        most[c["op"]] = max(most.get(c["op"], 0.0), w["bytes"] / 6.7e12 + w["flops"] / 1.9e15)
    op = rng.choice(["rope", "write", "read", "attend", "attend", "beam"])
    while True:
        dim = rng.choice([64, 96, 128, 128])
        heads = rng.choice([1, 2, 3, 4, 8])
        dtype = rng.choice(["bf16", "fp16"])
        fmt = rng.choice(["e4m3", dtype])
        page = rng.choice([16, 32, 64, 128])
        batch = _spread(rng, 1, 32)
        if op == "rope":
            c = dict(op=op, n=_spread(rng, 1, 8192), heads=rng.randint(1, 40), dim=dim,
                     rot=rng.choice([dim, dim // 2, 32]), interleaved=rng.random() < 0.5,
                     dtype=rng.choice(["bf16", "fp16", "fp32"]), scaled=rng.random() < 0.5,
                     far=_spread(rng, 16, 1 << 20), grad=rng.random() < 0.5)
        elif op == "write":
            c = dict(op=op, batch=batch, tokens=_spread(rng, 1, 2048), kv_heads=heads, dim=dim,
                     rot=rng.choice([dim, dim // 2]), interleaved=rng.random() < 0.5, dtype=dtype, fmt=fmt, page=page,
                     ctx=_spread(rng, 1, 8192) - 1, ragged=rng.random() < 0.5)
        elif op == "read":
            c = dict(op=op, batch=batch, kv_heads=heads, dim=dim, dtype=dtype, fmt=fmt, page=page,
                     ctx=_spread(rng, 1, 16384), ragged=rng.random() < 0.5)
        elif op == "attend":
            c = dict(op=op, batch=batch, tokens=rng.choice([1, 1, _spread(rng, 2, 64)]), kv_heads=heads,
                     group=rng.choice([1, 2, 4, 5, 7, 8]), dim=dim, dtype=dtype, fmt=fmt, page=page,
                     ctx=_spread(rng, 1, 98304), mask=rng.choice(["chain", "tree", "block"]),
                     ragged=rng.random() < 0.5)
        else:
            beams = _spread(rng, 1, 16)
            c = dict(op=op, batch=_spread(rng, 1, 16), beams=beams, vocab=_spread(rng, 100, 151936),
                     top=rng.choice([beams, 2 * beams]), states=rng.choice([0, 5, 64, 512]),
                     dead=rng.choice([0.5, 0.7, 0.9, 0.99]), dtype=rng.choice(["bf16", "fp16", "fp32"]),
                     length=_spread(rng, 8, 512))
        w = work(c)
        if w["bytes"] / 6.7e12 + w["flops"] / 1.9e15 <= most[op]:
            return c


def _lengths(c):
    """The cached length of each sequence: all `ctx`, or ragged down to an empty one."""
    B, n = c["batch"], c["ctx"]
    if not c["ragged"]:
        return [n] * B
    out = [max(0, n * (B - b) // B - (5 * b) % 7) for b in range(B)]
    if B > 3:
        out[-1] = 0
    return out


def _drafted(c):
    """How many drafted tokens of each sequence are in use."""
    T = c["tokens"]
    return [max(1, T - b % 3) if c["ragged"] else T for b in range(c["batch"])]


def work(case):
    """Bytes and operations that one pass cannot do without."""
    c = case
    if c["op"] == "rope":
        once = 2.0 * c["n"] * c["heads"] * c["dim"] * ES[c["dtype"]]
        both = 2 if c["grad"] else 1
        return {"bytes": both * once + 4.0 * c["n"], "flops": both * 3.0 * c["n"] * c["heads"] * c["rot"]}
    if c["op"] == "beam":
        cells = float(c["batch"]) * c["beams"] * c["vocab"]
        mask = cells / 8 if c["states"] else 0.0
        return {"bytes": cells * ES[c["dtype"]] + mask + 8.0 * c["batch"] * c["top"] * c["length"], "flops": 2 * cells}
    token = 2.0 * c["kv_heads"] * c["dim"]  # key and value elements of a token
    scale = 8.0 * c["kv_heads"] if c["fmt"] == "e4m3" else 0.0
    if c["op"] == "write":
        n = float(sum(_drafted(c)))
        return {"bytes": n * (token * (ES[c["dtype"]] + ES[c["fmt"]]) + scale), "flops": n * 4 * token}
    if c["op"] == "read":
        n, padded = float(sum(_lengths(c))), float(c["batch"] * c["ctx"])
        return {"bytes": n * (token * ES[c["fmt"]] + scale) + padded * token * ES[c["dtype"]], "flops": n * token}
    keys = [n + t for n, t in zip(_lengths(c), _drafted(c))]
    rows = c["kv_heads"] * c["group"]
    return {"bytes": sum(keys) * (token * ES[c["fmt"]] + scale) +
            2.0 * c["batch"] * c["tokens"] * rows * c["dim"] * ES[c["dtype"]],
            "flops": 4.0 * c["dim"] * rows * sum(k * t for k, t in zip(keys, _drafted(c)))}


# ------------------------------------------------------------------ inputs

def _phases(c, rot):
    """The angle of each rotated pair per position, in turns as a 64-bit fixed-point fraction
    (an int64 holding the bits): base 10000, stretched by 8 where the case is scaled."""
    got = []
    for i in range(rot // 2):
        turns = 10000.0 ** (-2.0 * i / rot) / (2 * math.pi) / (8.0 if c.get("scaled") else 1.0)
        bits = int(turns * 2.0 ** 64) % (1 << 64)
        got.append(bits - (1 << 64) if bits >= 1 << 63 else bits)
    return torch.tensor(got, dtype=torch.int64, device="cuda")


def _mscale(c):
    return 0.1 * math.log(8.0) + 1.0 if c.get("scaled") else 1.0


def _pages(c, gen, slots):
    """A page table over a pool with a few pages to spare, in no order."""
    per = max(1, -(-slots // c["page"]))
    n = c["batch"] * per + 3
    order = torch.randperm(n, generator=gen, device="cuda")[:c["batch"] * per]
    return n, order.to(torch.int32).view(c["batch"], per)


def _pool(c, gen, n_pages, fill):
    """Key and value pages with their scales, empty or filled as after earlier writes."""
    shape = (n_pages, c["kv_heads"], c["page"], c["dim"])
    got = {}
    for name in ("k", "v"):
        if c["fmt"] == "e4m3":
            if fill:
                x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)
                scale = x.abs().amax(-1) / E4M3_MAX
                got[name] = (x / scale[..., None]).to(torch.float8_e4m3fn)
                got[name + "_scale"] = scale
            else:
                got[name] = torch.zeros(shape, device="cuda", dtype=torch.uint8).view(torch.float8_e4m3fn)
                got[name + "_scale"] = torch.zeros(shape[:3], device="cuda", dtype=torch.float32)
        else:
            got[name] = torch.randn(shape, generator=gen, device="cuda").to(DT[c["fmt"]]) if fill else \
                torch.zeros(shape, device="cuda", dtype=DT[c["fmt"]])
            got[name + "_scale"] = None
    return got


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _tree_words(c, seed):
    """Which drafted tokens each drafted token sees, as 64-bit words: None = all of them."""
    B, T = c["batch"], c["tokens"]
    if c["mask"] == "block":
        return None
    import random
    rng = random.Random(seed)
    words = -(-T // 64)
    rows = []
    for _ in range(B):
        seen = []
        for j in range(T):
            parent = j - 1 if c["mask"] == "chain" else rng.randint(-1, j - 1) if j else -1
            seen.append((seen[parent] if parent >= 0 else 0) | 1 << j)
        rows.append([[_signed(s >> 64 * w & (1 << 64) - 1) for w in range(words)] for s in seen])
    return torch.tensor(rows, dtype=torch.int64, device="cuda")


def _signed(word):
    return word - (1 << 64) if word >= 1 << 63 else word


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)

    s = {"case": c}
    if c["op"] == "rope":
        dt = DT[c["dtype"]]
        s["x"] = normal(c["n"], c["heads"], c["dim"]).to(dt)
        s["out"] = torch.empty_like(s["x"])
        if c["grad"]:
            s["g"] = normal(c["n"], c["heads"], c["dim"]).to(dt)
            s["gx"] = torch.empty_like(s["x"])
        s["pos"] = torch.randint(0, c["far"], (c["n"],), generator=gen, device="cuda", dtype=torch.int32)
        s["phase"] = _phases(c, c["rot"])
    elif c["op"] == "write":
        B, T = c["batch"], c["tokens"]
        qkv = normal(B, T, 3 * c["kv_heads"], c["dim"]).to(DT[c["dtype"]])  # as a fused projection leaves them
        s["key"], s["value"] = qkv[:, :, c["kv_heads"]:2 * c["kv_heads"]], qkv[:, :, 2 * c["kv_heads"]:]
        n, s["table"] = _pages(c, gen, c["ctx"] + T)
        s.update(_pool(c, gen, n, False))
        s["start"], s["count"] = _ints(_lengths(c)), _ints(_drafted(c))
        s["pos"] = (s["start"][:, None] + torch.arange(T, device="cuda", dtype=torch.int32)).contiguous()
        s["phase"] = _phases(c, c["rot"])
    elif c["op"] == "read":
        n, s["table"] = _pages(c, gen, c["ctx"])
        s.update(_pool(c, gen, n, True))
        s["length"] = _ints(_lengths(c))
        shape = (c["batch"], c["ctx"], c["kv_heads"], c["dim"])
        s["key"], s["value"] = (torch.empty(shape, device="cuda", dtype=DT[c["dtype"]]) for _ in range(2))
    elif c["op"] == "attend":
        B, T, H = c["batch"], c["tokens"], c["kv_heads"] * c["group"]
        s["q"] = (1.5 * normal(B, T, H, c["dim"])).to(DT[c["dtype"]])
        n, s["table"] = _pages(c, gen, c["ctx"] + T)
        s.update(_pool(c, gen, n, True))
        s["length"], s["count"] = _ints(_lengths(c)), _ints(_drafted(c))
        s["mask"] = _tree_words(c, seed)
        if own:  # the workspace and the outputs that a program keeps from step to step
            from constrained_decoding_diffusion_gb300 import lm
            s["attend"] = lm.TreeAttention(B, T, H, c["kv_heads"], c["dim"], DT[c["dtype"]])
    else:
        N, K, V, S = c["batch"], c["beams"], c["vocab"], c["states"]
        x = 3 * normal(N, K, V)
        x[..., V - V // 50:] = -math.inf  # the padded end of a vocabulary
        s["logp"] = torch.log_softmax(x, -1).to(DT[c["dtype"]])
        s["scores"] = -20 - 5 * normal(N, K).abs()
        s["history"] = torch.randint(0, V, (N, K, c["length"]), generator=gen, device="cuda", dtype=torch.int32)
        s["step"] = c["length"] // 2
        if S:
            to = torch.randint(0, S, (S, V), generator=gen, device="cuda", dtype=torch.int16)
            dead = torch.rand((S, V), generator=gen, device="cuda") < c["dead"]
            s["next"] = to.masked_fill_(dead, -1)
            bits = torch.zeros((S, -(-V // 32) * 32), dtype=torch.int32, device="cuda")
            bits[:, :V] = (s["next"] >= 0).to(torch.int32)
            place = torch.arange(32, device="cuda", dtype=torch.int32)
            s["live"] = torch.bitwise_left_shift(bits.view(S, -1, 32), place).sum(-1, dtype=torch.int32)
            s["state"] = torch.randint(0, S, (N, K), generator=gen, device="cuda", dtype=torch.int32)
        if own:
            from constrained_decoding_diffusion_gb300 import lm
            s["select"] = lm.BeamSelect(N, K, V, c["top"], DT[c["dtype"]])
            s["moved"] = torch.empty((N, c["top"], c["length"]), dtype=torch.int32, device="cuda")
    return s


# ------------------------------------------------------------------ one pass

def run(state):
    return (_own if own else _plain)[state["case"]["op"]](state, state["case"])


# -- the plain forms

def _turned(x, pos, phase, c, inverse):
    """x [..., heads, dim] in 32 bits, rotated at pos [...]."""
    rot, half = c["rot"], c["rot"] // 2
    turns = pos.long()[..., None] * phase  # wraps around: whole turns drop out
    angle = (turns >> 32).float() * (2 * math.pi / 2 ** 32)
    cos, sin = torch.cos(angle)[..., None, :], torch.sin(angle)[..., None, :]
    if inverse:
        sin = -sin
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if c["interleaved"] else (x[..., :half], x[..., half:rot])
    m = _mscale(c)
    p, q = (a * cos - b * sin) * m, (a * sin + b * cos) * m
    both = torch.stack([p, q], -1).flatten(-2) if c["interleaved"] else torch.cat([p, q], -1)
    return torch.cat([both, x[..., rot:]], -1)


def _plain_rope(s, c):
    out = _turned(s["x"].float(), s["pos"], s["phase"], c, False).to(s["x"].dtype)
    if not c["grad"]:
        return out
    return {"out": out, "grad": _turned(s["g"].float(), s["pos"], s["phase"], c, True).to(s["x"].dtype)}


def _slots(s, c, first, T):
    """The page and the place in it of T slots from `first`, for each sequence."""
    slot = first.long()[:, None] + torch.arange(T, device="cuda")
    per = s["table"].shape[1]
    page = torch.gather(s["table"].long(), 1, (slot // c["page"]).clamp(max=per - 1))
    return page, slot % c["page"]


def _plain_write(s, c):
    T = c["tokens"]
    key = _turned(s["key"].float(), s["pos"], s["phase"], c, False)
    page, place = _slots(s, c, s["start"], T)
    use = torch.arange(T, device="cuda")[None] < s["count"][:, None]
    page, place = page[use], place[use]
    for name, x in (("k", key[use]), ("v", s["value"].float()[use])):
        if c["fmt"] == "e4m3":
            scale = x.abs().amax(-1) / E4M3_MAX
            code = (x / torch.where(scale > 0, scale, 1.0)[..., None]).to(torch.float8_e4m3fn)
            s[name].view(torch.uint8)[page, :, place] = code.view(torch.uint8)
            s[name + "_scale"][page, :, place] = scale
        else:
            s[name][page, :, place] = x.to(s[name].dtype)
    return _written(s, c)


def _written(s, c):
    if c["fmt"] == "e4m3":
        return {"k": s["k"], "v": s["v"], "k_scale": s["k_scale"], "v_scale": s["v_scale"]}
    return {"k": s["k"], "v": s["v"]}


def _values(s, name, c):
    """The pages of every sequence in 32 bits: [batch, heads, slots, dim]."""
    table = s["table"].long()
    if c["fmt"] == "e4m3":
        x = s[name].view(torch.uint8)[table].view(torch.float8_e4m3fn).float()
        x = x * s[name + "_scale"][table][..., None]
    else:
        x = s[name][table].float()
    B, P, H, G, D = x.shape
    return x.permute(0, 2, 1, 3, 4).reshape(B, H, P * G, D)


def _plain_read(s, c):
    use = (torch.arange(c["ctx"], device="cuda")[None] < s["length"][:, None])[..., None, None]
    got = {}
    for name in ("k", "v"):
        x = _values(s, name, c)[:, :, :c["ctx"]].transpose(1, 2)
        got[name] = torch.where(use, x, 0.0).to(DT[c["dtype"]])
    return got


def _visible(s, c, slots):
    """Which slots each drafted token sees: [batch, tokens, slots]."""
    B, T = c["batch"], c["tokens"]
    at = torch.arange(slots, device="cuda")[None, None]
    n, use = s["length"][:, None, None], s["count"][:, None, None]
    j = (at - n).clamp(0, T - 1).expand(B, T, slots)
    if s["mask"] is None:
        tree = torch.ones((B, T, slots), dtype=torch.bool, device="cuda")
    else:
        place = torch.arange(T, device="cuda")
        bits = (s["mask"][:, :, place // 64] >> (place % 64)) & 1
        tree = torch.gather(bits, 2, j) != 0
    row = torch.arange(T, device="cuda")[None, :, None] < use
    return row & ((at < n) | ((at < n + use) & tree))


def _plain_attend(s, c):
    B, T, H, G, D = c["batch"], c["tokens"], c["kv_heads"], c["group"], c["dim"]
    key, value = _values(s, "k", c), _values(s, "v", c)
    q = s["q"].float().view(B, T, H, G, D).permute(0, 2, 1, 3, 4).reshape(B, H, T * G, D)
    sees = _visible(s, c, key.shape[2])[:, None].repeat_interleave(G, 2)
    x = torch.matmul(q, key.transpose(2, 3)) * (1.0 / math.sqrt(D))
    x = torch.where(sees, x, -math.inf)
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(top > -math.inf, top, 0.0))
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p, value) / torch.where(total > 0, total, 1.0)
    lse = (top + torch.log(total)).squeeze(-1)
    out = out.view(B, H, T, G, D).permute(0, 2, 1, 3, 4).reshape(B, T, H * G, D).to(s["q"].dtype)
    return {"out": out, "lse": lse.view(B, H, T, G).permute(0, 2, 1, 3).reshape(B, T, H * G)}


def _plain_beam(s, c):
    N, K, V, top = c["batch"], c["beams"], c["vocab"], c["top"]
    x = s["scores"][..., None] + s["logp"].float()
    ok = x > -math.inf  # false for NaN too
    if c["states"]:
        ok = ok & (s["next"][s["state"].long()] >= 0)
    best, at = torch.sort(torch.where(ok, x, -math.inf).view(N, K * V), dim=-1, descending=True, stable=True)
    score, at = best[:, :top], at[:, :top]
    if score.shape[1] < top:  # fewer cells than were asked for
        score = torch.nn.functional.pad(score, (0, top - score.shape[1]), value=-math.inf)
        at = torch.nn.functional.pad(at, (0, top - at.shape[1]))
    found = score > -math.inf
    parent, token = torch.where(found, at // V, -1), torch.where(found, at % V, -1)
    got = {"score": score, "parent": parent.int(), "token": token.int()}
    up = parent.clamp(min=0)
    if c["states"]:
        old = torch.gather(s["state"].long(), 1, up)
        got["state"] = torch.where(found, s["next"][old, token.clamp(min=0)].long(), -1).int()
    moved = torch.gather(s["history"], 1, up[..., None].expand(-1, -1, c["length"]))
    moved = torch.where(found[..., None], moved, -1)
    moved[..., s["step"]] = token.int()
    got["history"] = moved
    return got


_plain = {"rope": _plain_rope, "write": _plain_write, "read": _plain_read, "attend": _plain_attend,
          "beam": _plain_beam}


# -- the package's calls

def _own_rope(s, c):
    from constrained_decoding_diffusion_gb300 import lm
    more = dict(interleaved=c["interleaved"], mscale=_mscale(c))
    out = lm.fa_rope(s["x"], s["pos"], s["phase"], out=s["out"], **more)
    if not c["grad"]:
        return out
    return {"out": out, "grad": lm.fa_rope(s["g"], s["pos"], s["phase"], out=s["gx"], inverse=True, **more)}


def _cache(s, lm):
    return lm.KVCache(s["k"], s["v"], s["k_scale"], s["v_scale"])


def _own_write(s, c):
    from constrained_decoding_diffusion_gb300 import lm
    lm.fa_cache_write(_cache(s, lm), s["key"], s["value"], s["table"], s["start"], count=s["count"],
                      positions=s["pos"], phase=s["phase"], interleaved=c["interleaved"])
    return _written(s, c)


def _own_read(s, c):
    from constrained_decoding_diffusion_gb300 import lm
    lm.fa_cache_read(_cache(s, lm), s["table"], s["length"], s["key"], s["value"])
    return {"k": s["key"], "v": s["value"]}


def _own_attend(s, c):
    from constrained_decoding_diffusion_gb300 import lm
    out, lse = s["attend"](s["q"], _cache(s, lm), s["table"], s["length"], mask=s["mask"], count=s["count"])
    return {"out": out, "lse": lse}


def _own_beam(s, c):
    from constrained_decoding_diffusion_gb300 import lm
    if c["states"]:
        score, parent, token, state = s["select"](s["logp"], s["scores"], s["state"], s["next"], s["live"])
        got = {"score": score, "parent": parent, "token": token, "state": state}
    else:
        score, parent, token, _ = s["select"](s["logp"], s["scores"])
        got = {"score": score, "parent": parent, "token": token}
    got["history"] = lm.fa_beam_reorder(s["history"], parent, s["moved"], token=token, at=s["step"])
    return got


_own = {"rope": _own_rope, "write": _own_write, "read": _own_read, "attend": _own_attend, "beam": _own_beam}


# ------------------------------------------------------------------ the definitions in 64 bits

def _rotation(x, pos, c, inverse):
    """One pair at a time: the pair's two elements as a complex number times exp(i angle)."""
    out = x.double().clone()
    rot = c["rot"]
    for i in range(rot // 2):
        w = 10000.0 ** (-2.0 * i / rot) / (8.0 if c.get("scaled") else 1.0)
        turn = torch.polar(torch.full(pos.shape, _mscale(c), dtype=torch.float64, device="cuda"),
                           pos.double() * (-w if inverse else w))[..., None]
        a, b = (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + rot // 2)
        z = torch.complex(x[..., a].double(), x[..., b].double()) * turn
        out[..., a], out[..., b] = z.real, z.imag
    return out


def _nearest_e4m3(x):
    """The 8-bit floating value nearest to each x in [-448, 448], ties to even."""
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(x / step) * step


def _sequence(s, name, c, b, n):
    """The first n cached rows of a sequence: [n, heads, dim] in 64 bits."""
    rows = []
    for p in range(-(-n // c["page"])):
        at = int(s["table"][b, p])
        x = s[name][at].double()
        if c["fmt"] == "e4m3":
            x = x * s[name + "_scale"][at].double()[..., None]
        rows.append(x.transpose(0, 1))
    return torch.cat(rows)[:n] if rows else torch.zeros((0, c["kv_heads"], c["dim"]), dtype=torch.float64, device="cuda")


def exact(case, seed):
    c = case
    s = prepare(c, seed)
    if c["op"] == "rope":
        out = _rotation(s["x"], s["pos"], c, False)
        return {"out": out, "grad": _rotation(s["g"], s["pos"], c, True)} if c["grad"] else out
    if c["op"] == "write":
        key = _rotation(s["key"], s["pos"], c, False)
        got = {}
        for name, x in (("k", key), ("v", s["value"].double())):
            pages = s[name].double()
            scales = s[name + "_scale"].double() if c["fmt"] == "e4m3" else None
            for b, (n, use) in enumerate(zip(_lengths(c), _drafted(c))):
                slot = torch.arange(n, n + use, device="cuda")
                page, place = s["table"][b].long()[slot // c["page"]], slot % c["page"]
                rows = x[b, :use]
                if scales is not None:
                    scale = rows.abs().amax(-1) / E4M3_MAX
                    scales[page, :, place] = scale
                    rows = _nearest_e4m3(rows / scale[..., None])
                pages[page, :, place] = rows
            got[name] = pages
            if scales is not None:
                got[name + "_scale"] = scales
        return got
    if c["op"] == "read":
        got = {}
        for name in ("k", "v"):
            x = torch.zeros(s["key"].shape, dtype=torch.float64, device="cuda")
            for b, n in enumerate(_lengths(c)):
                x[b, :n] = _sequence(s, name, c, b, n)
            got[name] = x
        return got
    if c["op"] == "attend":
        B, T, H, G, D = c["batch"], c["tokens"], c["kv_heads"], c["group"], c["dim"]
        out = torch.zeros((B, T, H * G, D), dtype=torch.float64, device="cuda")
        lse = torch.full((B, T, H * G), -math.inf, dtype=torch.float64, device="cuda")
        words = None if s["mask"] is None else s["mask"].cpu().tolist()
        for b, (n, use) in enumerate(zip(_lengths(c), _drafted(c))):
            key, value = _sequence(s, "k", c, b, n + use), _sequence(s, "v", c, b, n + use)
            sees = torch.ones((use, n + use), dtype=torch.bool)
            if words is not None:
                for i in range(use):
                    for j in range(use):
                        sees[i, n + j] = bool(words[b][i][j // 64] >> (j % 64) & 1)
            sees = sees.cuda()
            for h in range(H):
                q = s["q"][b, :use, h * G:(h + 1) * G].double()
                x = torch.einsum("tgd,nd->tgn", q, key[:, h]) / math.sqrt(D)
                x = x.masked_fill(~sees[:, None], -math.inf)
                lse[b, :use, h * G:(h + 1) * G] = torch.logsumexp(x, -1)
                out[b, :use, h * G:(h + 1) * G] = torch.einsum("tgn,nd->tgd", torch.softmax(x, -1), value[:, h])
        return {"out": out, "lse": lse}
    N, K, V = c["batch"], c["beams"], c["vocab"]
    score = torch.full((N, c["top"]), -math.inf, dtype=torch.float64, device="cuda")
    for n in range(N):
        x = s["scores"][n].double()[:, None] + s["logp"][n].double()
        if c["states"]:
            x = x.masked_fill(s["next"][s["state"][n].long()] < 0, -math.inf)
        best = torch.topk(x.flatten(), min(c["top"], K * V)).values
        score[n, :best.numel()] = best
    return {"score": score, "parent": None, "token": None, "state": None, "history": None}
