"""The rotary function's derivatives of every order.  On the CPU the library's call is stood in for by one
that, like it, fills a new tensor without a graph; on the GPU it is the call itself."""
import math

import pytest

torch = pytest.importorskip("torch")

from constrained_decoding_diffusion_gb300 import lm  # noqa: E402


def plain(x, positions, phase, interleaved=False, mscale=1.0, inverse=False):
    half = phase.numel()
    angle = positions.double()[:, None] * (phase.double() * (2 * math.pi / 2.0 ** 64)) * (-1 if inverse else 1)
    c, s = ((mscale * f(angle))[:, None].to(x.dtype) for f in (torch.cos, torch.sin))
    rot = x[..., :2 * half]
    a, b = (rot[..., ::2], rot[..., 1::2]) if interleaved else (rot[..., :half], rot[..., half:])
    p, q = a * c - b * s, a * s + b * c
    both = torch.stack((p, q), -1).flatten(-2) if interleaved else torch.cat((p, q), -1)
    return torch.cat((both, x[..., 2 * half:]), -1)


def inputs(device, dtype):
    g = torch.Generator().manual_seed(3)
    x, w = (torch.randn((3, 2, 10), generator=g, dtype=dtype).to(device) for _ in range(2))
    phase, _ = lm.rope_phases(8, device=device)
    return x, w, torch.tensor([0, 5, 70001], dtype=torch.int32, device=device), phase


@pytest.mark.parametrize("interleaved", [False, True])
def test_derivatives_against_differences(monkeypatch, interleaved):
    def stand_in(x, positions, phase, out=None, interleaved=False, mscale=1.0, inverse=False, stream=None):
        with torch.no_grad():
            return plain(x, positions, phase, interleaved, mscale, inverse).clone()
    monkeypatch.setattr(lm, "fa_rope", stand_in)
    x, _, pos, phase = inputs("cpu", torch.float64)
    x.requires_grad_(True)

    def f(y):
        return torch.sin(lm.Rope.apply(y, pos, phase, interleaved, 1.25))
    assert torch.autograd.gradcheck(f, x)
    assert torch.autograd.gradgradcheck(f, x)


@pytest.mark.gpu
@pytest.mark.parametrize("interleaved", [False, True])
def test_second_derivative(interleaved):
    """A gradient's penalty, |d f / d x|^2, differentiated through the library's calls and through torch's.
    Values of order one through two rotations in fp32 and a cube: 1e-4 is far above their rounding and far
    below a lost term."""
    got = []
    for rotate in (lambda y: lm.Rope.apply(y, pos, phase, interleaved, 1.25), lambda y: plain(y, pos, phase, interleaved, 1.25)):
        x, w, pos, phase = inputs("cuda", torch.float32)
        x.requires_grad_(True)
        first, = torch.autograd.grad((w * rotate(x) ** 3).sum(), x, create_graph=True)
        second, = torch.autograd.grad((first ** 2).sum(), x)
        got.append((first.detach(), second))
    for a, b in zip(*got):
        assert (a - b).abs().max() <= 1e-4 * b.abs().max()
