"""Verification of drafted tokens against the definition in 64 bits.  Every output is a whole number; a draw within
2^-46 of a border between two tokens could go either way, which the chosen numbers do not meet."""
import pytest

torch = pytest.importorskip("torch")

import serving_reference as ref  # noqa: E402
from constrained_decoding_diffusion_gb300 import lm  # noqa: E402

pytestmark = pytest.mark.gpu

F32, BF, HF = torch.float32, torch.bfloat16, torch.float16


def chain(T):
    return list(range(-1, T - 1))


def beams(K, depth):
    return [-1] + [0 if (j - 1) % depth == 0 else j - 1 for j in range(1, 1 + K * depth)]


def automaton(g, S, V, dead=0.6):
    nxt = torch.randint(0, S, (S, V), generator=g, dtype=torch.int16)
    nxt[torch.rand(S, V, generator=g) < dead] = -1
    bits = torch.zeros(S, -(-V // 32) * 32, dtype=torch.int64)
    bits[:, :V] = nxt >= 0
    words = (bits.view(S, -1, 32) << torch.arange(32)).sum(-1)
    return nxt.cuda(), (words - (words >> 31 << 32)).int().cuda()


def make(seed, B, parents, V, dtype=F32, draft=True, states=0, spread=3.0, sampled=True):
    g = torch.Generator().manual_seed(seed)
    T = len(parents)
    x = spread * torch.randn(B, T, V, generator=g)
    d = dict(target=torch.softmax(x + torch.randn(B, T, V, generator=g), -1).to(dtype).cuda(),
             parents=torch.tensor([parents] * B, dtype=torch.int32).cuda(), u=torch.rand(B, T, generator=g).cuda())
    up = torch.tensor(parents).clamp(min=0)
    rows = torch.softmax(x, -1)[:, up]
    tokens = torch.multinomial(rows.view(B * T, V), 1, generator=g).view(B, T) if sampled else rows.argmax(-1)
    d["tokens"] = tokens.int().cuda()
    if draft:
        d["draft"] = torch.softmax(x, -1).to(dtype).cuda()
    if states:
        d["next"], d["live"] = automaton(g, states, V)
        d["states"] = torch.randint(0, states, (B,), generator=g, dtype=torch.int32).cuda()
    return d


def check(d, call=None):
    B, T, V = d["target"].shape
    call = call or lm.Verify(B, T, V, d["target"].dtype)
    for x in (call.path, call.kept, call.token, call.state):
        x.fill_(-7)
    got = call(**d)
    want = ref.verify(d["target"], d["tokens"], d["parents"], d["u"], d.get("draft"), d.get("count"), d.get("states"), d.get("next"))
    for name, g, w in zip(("path", "kept", "token", "state"), got, want):
        if g is not None:
            assert (g.cpu().numpy() == w).all(), name
    return [None if x is None else x.clone() for x in got]


@pytest.mark.parametrize("dtype", [F32, HF, BF])
@pytest.mark.parametrize("V", [1, 2, 7, 31, 33, 100, 1000, 4097, 33333])
@pytest.mark.parametrize("draft,states", [(True, 0), (False, 0), (True, 5), (False, 5)])
def test_chains_and_trees(dtype, V, draft, states):
    """Odd vocabularies leave the rows unaligned; the numbers of the nodes are in the order of the beams."""
    check(make(V, 6, chain(5), V, dtype, draft, states))
    check(make(V + 1, 5, beams(3, 3), V, dtype, draft, states))


@pytest.mark.parametrize("draft", [True, False])
@pytest.mark.parametrize("T", [1, 2, 40, 1024])
def test_lengths_of_drafts(T, draft):
    check(make(T, 3, chain(T), 50, draft=draft, spread=1.0))
    check(make(T, 2, [-1] + [0] * (T - 1), 50, draft=draft, spread=1.0))   # many children of one node


def test_random_trees_and_parents_that_are_none():
    g = torch.Generator().manual_seed(3)
    for seed in range(8):
        d = make(seed, 4, chain(24), 300, draft=seed % 2 == 0, spread=1.5)
        parents = (torch.rand(4, 24, generator=g) * torch.arange(24)).int() - 1
        parents[:, 5] = 5
        parents[:, 6] = 9
        parents[0, 1:] = -1
        d["parents"] = parents.cuda()
        check(d)


def test_same_token_twice_among_siblings():
    for draft in (True, False):
        d = make(11, 8, [-1, 0, 0, 0, 0, 1, 1], 20, draft=draft, spread=1.0)
        d["tokens"][:, 2] = d["tokens"][:, 1]
        d["tokens"][:, 6] = d["tokens"][:, 5]
        check(d)


@pytest.mark.parametrize("draft", [True, False])
def test_tokens_that_are_none(draft):
    d = make(5, 4, beams(2, 3), 64, draft=draft)
    d["tokens"][:, 1] = -1
    d["tokens"][1, 4] = 64
    d["tokens"][2] = torch.iinfo(torch.int32).min
    d["tokens"][3] = torch.iinfo(torch.int32).max
    check(d)


@pytest.mark.parametrize("draft,states", [(True, 0), (False, 6)])
def test_counts(draft, states):
    d = make(6, 7, chain(6), 500, draft=draft, states=states)
    d["count"] = torch.tensor([0, 1, 2, 6, 100, -3, 4], dtype=torch.int32).cuda()
    check(d)


@pytest.mark.parametrize("V", [40, 9001])
@pytest.mark.parametrize("draft", [True, False])
def test_odd_weights(draft, V):
    """What is not a positive finite number has no weight, and rows need not add up to one."""
    d = make(8, 6, beams(2, 2), V, draft=draft, spread=1.0)
    g = torch.Generator().manual_seed(1)
    for name in ("target", "draft"):
        if name in d:
            for i, v in enumerate((float("nan"), float("inf"), -1.0, 0.0, -float("inf"), 1e-42)):
                d[name][i][(torch.rand(5, V, generator=g) < 0.3).cuda()] = v
            d[name][1] *= 1000.0
            d[name][2] *= 2.0 ** -40
    check(d)


@pytest.mark.parametrize("draft", [True, False])
def test_rows_without_weight(draft):
    d = make(9, 4, chain(3), 5000, draft=draft)
    d["target"][0] = 0
    d["target"][1, 1:] = 0
    d["target"][2, 0] = 0
    d["target"][2, 0, 4999] = 1e-30
    if draft:
        d["draft"][3] = 0
    path, kept, token, _ = check(d)
    assert token[0] == -1 and kept[0] == 1


@pytest.mark.parametrize("draft", [True, False])
@pytest.mark.parametrize("V", [50, 9001])
def test_sums_beyond_fp32(draft, V):
    """A target row whose sum leaves fp32 has no token; a draft row whose sum does accepts nothing that the target's lacks,
    and its sequence still ends with a token."""
    d = make(19, 3, chain(3), V, draft=draft)
    d["target"][0, 0] = 3e38
    if draft:
        d["draft"][1] = 3e38
    path, kept, token, _ = lm.Verify(3, 3, V)(**d)
    assert token[0] == -1 and kept[0] == 1 and path[0].tolist() == [0, -1, -1]
    assert ((token[1:] >= 0) & (token[1:] < V)).all() and ((kept[1:] >= 1) & (kept[1:] <= 3)).all()


def test_states_outside_and_dead():
    d = make(10, 6, chain(4), 700, states=4)
    d["states"] = torch.tensor([-1, 4, 0, 1, 2, 3], dtype=torch.int32).cuda()
    d["next"][2] = -1
    d["live"][2] = 0
    path, kept, token, state = check(d)
    assert token[:2].tolist() == [-1, -1] and state[4] == -1


@pytest.mark.parametrize("draft", [True, False])
@pytest.mark.parametrize("u", [0.0, 1.0 - 2.0 ** -24, 1.0, float("nan"), -1.0])
def test_borders_of_the_numbers(u, draft):
    d = make(12, 3, beams(2, 2), 3001, draft=draft)
    d["u"].fill_(u)
    if u in (0.0, 1.0 - 2.0 ** -24):
        check(d)
        return
    d["u"][:, 0] = 0.5                     # outside [0, 1): nothing is accepted below 1, and nothing breaks
    path, kept, token, _ = lm.Verify(3, 5, 3001)(**d)
    assert ((token >= 0) & (token < 3001)).all() and ((kept >= 1) & (kept <= 3)).all()


def test_the_target_itself_as_draft_is_accepted():
    d = make(13, 5, chain(6), 2000)
    d["draft"] = d["target"]
    _, kept, _, _ = check(d)
    assert (kept == 6).all()


@pytest.mark.parametrize("dtype", [F32, BF])
def test_strides(dtype):
    """Rows of a wider buffer that start anywhere, one row for all nodes, rows in any order."""
    d = make(14, 3, chain(4), 6000, dtype, states=3)
    for lead in (0, 1, 3, 4):
        for name, more in (("target", 5), ("draft", 2)):
            wide = torch.full((3, 4, 6000 + lead + more), float("nan"), dtype=dtype, device="cuda")
            wide[..., lead:lead + 6000] = d[name]
            d[name] = wide[..., lead:lead + 6000]
        check(d)
    d["draft"] = d["draft"][:, :1].expand(3, 4, 6000)
    d["target"] = d["target"].transpose(0, 1).contiguous().transpose(0, 1)
    check(d)


@pytest.mark.parametrize("draft,states", [(True, 0), (False, 0), (False, 3)])
def test_first_token_has_the_targets_distribution(draft, states):
    """Over many numbers the token after node 0 (the first accepted one, or the next token) has the target's
    frequencies: of n draws, each frequency is within 5 sqrt(p (1 - p) / n)."""
    B, V, parents = 60000, 6, [-1, 0, 0, 1]
    g = torch.Generator().manual_seed(2)
    p = torch.tensor([0.3, 0.05, 0.2, 0.25, 0.1, 0.1])
    q = torch.tensor([0.05, 0.4, 0.1, 0.15, 0.1, 0.2])
    nxt = torch.zeros(max(states, 1), V, dtype=torch.int16)
    if states:
        nxt[0, 2] = -1
        p = torch.where(torch.arange(V) == 2, 0.0, p)
        p /= p.sum()
    tokens = torch.multinomial(q.expand(B, V), 4, replacement=True, generator=g).int()
    if not draft:
        tokens[:, 1], tokens[:, 2] = 1, 4
    d = dict(target=p.expand(B, 4, V).cuda(), tokens=tokens.cuda(),
             parents=torch.tensor(parents, dtype=torch.int32).expand(B, 4).contiguous().cuda(),
             u=torch.rand(B, 4, generator=g).cuda())
    if draft:
        d["draft"] = q.expand(B, 4, V).cuda()
    if states:
        d["next"] = nxt.cuda()
        d["live"] = ((nxt >= 0).long() << torch.arange(V)).sum(-1, keepdim=True).int().cuda()
        d["states"] = torch.zeros(B, dtype=torch.int32, device="cuda")
    path, kept, token, _ = lm.Verify(B, 4, V)(**d)
    first = torch.where(kept > 1, d["tokens"].gather(1, path[:, 1:2].clamp(min=0).long())[:, 0], token).cpu()
    seen = torch.bincount(first.long(), minlength=V) / B
    assert ((seen - p).abs() <= 5 * (p * (1 - p) / B).sqrt() + 1e-12).all()


def test_captured_and_on_another_stream():
    d = make(15, 9, beams(4, 3), 20011, states=7, draft=False, sampled=False)
    call = lm.Verify(9, 13, 20011)
    want = check(d, call)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    again = lm.Verify(9, 13, 20011)
    got = again(**d, stream=side)
    side.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call(**d)
    for seed in (16, 17):
        new = make(seed, 9, beams(4, 3), 20011, states=7, draft=False, sampled=False)
        for k in ("target", "tokens", "u", "states", "next", "live"):
            d[k].copy_(new[k])
        graph.replay()
        want = ref.verify(d["target"], d["tokens"], d["parents"], d["u"], None, None, d["states"], d["next"])
        assert all((g.cpu().numpy() == w).all() for g, w in zip(got, want))


def test_many_sequences_over_a_large_vocabulary():
    d = make(18, 40, chain(3), 70001, BF, states=2)
    first = check(d)
    assert all(torch.equal(x, y) for x, y in zip(first, check(d)))


@pytest.mark.parametrize("V", [4, 40000])
def test_a_sum_of_which_only_roundings_are_left(V):
    """Four tokens weigh 1, 2^-23, x and 3/4 of x's last place, x = 1.5 2^-47, and all are tried with the largest u.  As two
    floats the sum is 1 + 2^-23 + (x + 1 last place), so each is rejected, and a quarter of x's last place is left of
    nothing.  The next token is none rather than what the buffer held."""
    x, last = 1.5 * 2.0 ** -47, 2.0 ** -70
    target = torch.zeros(1, 5, V)
    target[0, 0, :4] = torch.tensor([1.0, x, 2.0 ** -23, 0.75 * last])
    verify = lm.Verify(1, 5, V)
    for out in (verify.path, verify.kept, verify.token):
        out.fill_(77)
    path, kept, token, _ = verify(target.cuda(), torch.tensor([[0, 0, 2, 1, 3]], dtype=torch.int32).cuda(),
                                  torch.tensor([[-1, 0, 0, 0, 0]], dtype=torch.int32).cuda(),
                                  torch.full((1, 5), 1 - 2.0 ** -24).cuda())
    assert path.tolist() == [[0, -1, -1, -1, -1]] and kept.tolist() == [1]
    assert token.tolist() == [-1]


@pytest.mark.parametrize("dtype,draft,states", [(F32, True, 0), (BF, False, 3), (HF, True, 3)])
@pytest.mark.parametrize("B,V", [(1, 98303), (1, 98304), (12, 98304), (13, 98311), (15, 122887), (16, 131075), (17, 131072)])
def test_large_vocabularies_of_few_sequences(B, V, dtype, draft, states):
    check(make(V + B, B, chain(3), V, dtype, draft, states))
    check(make(V, B, [-1, 0, 0, 0], V, dtype, draft, states, sampled=False))


def test_more_drafted_tokens_than_threads_over_a_large_vocabulary():
    """600 children of the last token, then a chain; a state's moves are looked up for all of them."""
    g = torch.Generator().manual_seed(2)
    d = make(3, 2, [-1] + [0] * 600, 5, draft=False)
    V = 98400
    d["target"] = torch.rand(2, 601, V, generator=g).cuda()
    d["tokens"] = torch.randperm(V, generator=g)[:1202].view(2, 601).int().cuda()
    d["u"][:, 1:] = 1 - 2.0 ** -20
    d["u"][1, 500] = 0.0
    d["next"], d["live"] = automaton(g, 4, V, dead=0.3)
    d["states"] = torch.tensor([1, 2], dtype=torch.int32).cuda()
    check(d)
