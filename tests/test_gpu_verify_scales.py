"""Verification of rows whose sums lie anywhere in fp32's range, each row in its own."""
import pytest

torch = pytest.importorskip("torch")

from constrained_decoding_diffusion_gb300 import lm  # noqa: E402
from test_gpu_verify import BF, F32, beams, chain, check, make  # noqa: E402

pytestmark = pytest.mark.gpu


def scaled(d, target, draft):
    """Powers of two on whole rows (bf16 has fp32's range): exact but for what falls below 2^-149."""
    for name, e in (("target", target), ("draft", draft)):
        if d.get(name) is not None:
            half = e // 2
            d[name] = (d[name].float() * 2.0 ** half * 2.0 ** (e - half)).to(d[name].dtype)
    return d


@pytest.mark.parametrize("target,draft", [(-90, 70), (70, -90), (-60, 100), (100, -100), (-100, -100), (120, 120), (-130, 0), (0, -130),
                                          (-41, 41), (33, -33), (-126, 126), (126, -126)])
@pytest.mark.parametrize("V", [40, 5003])
@pytest.mark.parametrize("dtype,states", [(F32, 0), (F32, 3), (BF, 0)])
def test_rows_of_any_scale(target, draft, V, dtype, states):
    """Whole trees with rejections at every scale of the two rows; the outputs are whole numbers."""
    for parents in (chain(5), [-1, 0, 0, 0, 0, 1, 2]):
        d = scaled(make(V, 12, parents, V, dtype, True, states, spread=1.5), target, draft)
        d["tokens"] = torch.roll(d["tokens"], 1, 0)            # another sequence's draws: many are rejected
        _, kept, _, _ = check(d)
        if dtype == F32 and not states:                        # (few rolled tokens are allowed, and bf16's small ones are zero)
            assert (kept == 1).any() and (kept > 1).any()


@pytest.mark.parametrize("target", [-120, -90, 90])
def test_scales_without_a_draft(target):
    check(scaled(make(3, 12, beams(3, 3), 5003, F32, False, spread=1.0), target, 0))


@pytest.mark.parametrize("V", [40, 5003])
@pytest.mark.parametrize("target", [-100, 0, 100])
def test_a_draft_whose_sum_is_beyond_fp32(V, target):
    """Its weights are finite, so the distribution that it stands for is there all the same."""
    d = scaled(make(7, 12, [-1, 0, 0, 1], V, spread=1.0), target, 0)
    g = torch.Generator().manual_seed(1)
    d["draft"] = torch.rand(12, 4, V, generator=g).cuda() * 3.4e38
    d["tokens"] = torch.randint(0, V, (12, 4), generator=g).int().cuda()
    _, kept, _, _ = check(d)
    assert (kept == 1).any() and (kept > 1).any()


def test_each_row_has_its_own_scale():
    d = make(9, 30, chain(6), 700, spread=1.0)
    g = torch.Generator().manual_seed(5)
    for name in ("target", "draft"):
        half = torch.randint(-50, 51, (30, 6, 1), generator=g).cuda()
        d[name] = d[name] * torch.exp2(half.float()) * torch.exp2(half.float())
    check(d)


@pytest.mark.parametrize("draft,states", [(True, 0), (True, 3), (False, 3)])
@pytest.mark.parametrize("B,V", [(3, 131075), (40, 98311)])
def test_scales_of_large_vocabularies(B, V, draft, states):
    """In sixteen blocks a sequence and in eight, with rows that start anywhere and a draft of another alignment."""
    d = scaled(make(V, B, [-1, 0, 0, 1], V, F32, draft, states), -100, 90)
    if draft:
        wide = torch.zeros(B, 4, V + 3, device="cuda")
        wide[..., 2:2 + V] = d["draft"]
        d["draft"] = wide[..., 2:2 + V]
    check(d)


def test_the_draw_follows_the_scaled_rows():
    """Of 60000 draws over rows whose sums are 2^-90 and 2^70, each frequency is within 5 sqrt(p (1 - p) / n)."""
    n, V = 60000, 6
    g = torch.Generator().manual_seed(2)
    p, q = torch.tensor([0.3, 0.05, 0.2, 0.25, 0.1, 0.1]), torch.tensor([0.05, 0.4, 0.1, 0.15, 0.1, 0.2])
    tokens = torch.multinomial(q.expand(n, V), 3, replacement=True, generator=g).int()
    path, kept, token, _ = (x if x is None else x.cpu() for x in lm.Verify(n, 3, V)(
        target=(p * 2.0 ** -90).expand(n, 3, V).cuda(), tokens=tokens.cuda(),
        parents=torch.tensor([[-1, 0, 0]] * n, dtype=torch.int32).cuda(), u=torch.rand(n, 3, generator=g).cuda(),
        draft=(q * 2.0 ** 70).expand(n, 3, V).cuda()))
    first = torch.where(kept > 1, tokens.gather(1, path[:, 1:2].clamp(min=0).long())[:, 0], token).long()
    seen = torch.bincount(first, minlength=V) / n
    assert ((seen - p).abs() <= 5 * (p * (1 - p) / n).sqrt()).all()
