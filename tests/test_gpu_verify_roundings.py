"""Draws of which rejections have left little: tokens without weight beside them, roundings in their place."""
import pytest

torch = pytest.importorskip("torch")

import serving_reference as ref  # noqa: E402
from constrained_decoding_diffusion_gb300 import lm  # noqa: E402
from test_gpu_serving_sizes import ints  # noqa: E402

pytestmark = pytest.mark.gpu


def small(V, where):
    """Weights 1, 2^-23, x and 3/4 of x's last place (x = 1.5 2^-47), whose rejections leave a rounding in their segment, and
    what else weighs."""
    target = torch.zeros(1, 5, V)
    target[0, :, :4] = torch.tensor([1.0, 1.5 * 2.0 ** -47, 2.0 ** -23, 0.75 * 2.0 ** -70])
    for v, w in where.items():
        target[0, :, v] = w
    return target


@pytest.mark.parametrize("u", [0.0, 2.0 ** -24, 0.25, 0.4375, 1 - 2.0 ** -24])
@pytest.mark.parametrize("where", [{39999: 0.5}, {20000: 0.25, 39999: 0.5}, {4: 0.5}, {39998: 2.0 ** -20, 39999: 2.0 ** -20},
                                   {700: 0.5, 701: 0.25}])
def test_weight_is_found_beside_roundings(where, u):
    """The four are all tried with the largest u and rejected (their shares are below it); what is left is drawn from, whatever
    rounding the segment of the four still holds."""
    V = 40000
    target = small(V, where)
    d = dict(target=target.cuda(), tokens=ints([[0, 0, 2, 1, 3]]), parents=ints([[-1, 0, 0, 0, 0]]),
             u=torch.tensor([[u] + [1 - 2.0 ** -24] * 4], device="cuda"))
    path, kept, token, _ = lm.Verify(1, 5, V)(**d)
    p, k, t, _ = ref.verify(d["target"], d["tokens"], d["parents"], d["u"])
    assert kept.tolist() == k.tolist() == [1] and path.cpu().numpy().tolist() == p.tolist()
    assert token.tolist() == t.tolist()


@pytest.mark.parametrize("V,at", [(40000, 39999), (40000, 9), (4097, 4096)])
def test_weight_below_the_sums_last_bits_is_found(V, at):
    """The only weight that has not been tried is 2^-100, below the last bits of the sum of those that have: it is the next token
    rather than none."""
    target = small(V, {at: 2.0 ** -100})
    for u in (0.0, 0.5, 1 - 2.0 ** -24):
        path, kept, token, _ = lm.Verify(1, 5, V)(
            target.cuda(), ints([[0, 0, 2, 1, 3]]), ints([[-1, 0, 0, 0, 0]]),
            torch.tensor([[u] + [1 - 2.0 ** -24] * 4], device="cuda"))
        assert kept.tolist() == [1] and token.tolist() == [at]
