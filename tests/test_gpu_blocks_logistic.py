"""The logistic function behind SiLU, GELU and a gate over its whole range: within its bound where
it is 2^-126 or more, 0 below."""
import pytest
import torch

from bit_microscaled_quantized_amd import blocks

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def near(got, arg, factor, roundings):
    """got against factor * p(arg): p within (5 + 1.25 |arg|) u of itself, `roundings` more; 0 below 2^-126 (either side of
    which p's own error decides)."""
    p = torch.sigmoid(arg)
    e = (5 + 1.25 * arg.abs()) * U
    want = p * factor
    inside, below = p >= 2.0 ** -126 * (1 + e), p < 2.0 ** -126 * (1 - e)
    assert bool(((got.double() - want).abs() <= want.abs() * (e + roundings * U))[inside].all())
    assert bool((got == 0)[below].all()) and int(below.sum()) > 100


def test_silu():
    v = torch.cat([torch.linspace(-120, 120, 240001), -torch.linspace(87.3, 87.4, 2001)]).cuda()
    with torch.no_grad():
        near(blocks.gated_act(v), v.double(), v.double(), 1)


def test_gelu():
    """Its argument has four roundings more (v^2, a factor, the sum, the product), each an error of |argument| u in p."""
    v = torch.linspace(-12, 12, 120001).cuda()
    d = v.double()
    arg = (8 / torch.pi) ** 0.5 * (d + 0.044715 * d ** 3)
    with torch.no_grad():
        y = blocks.gated_act(v, act="gelu")
    p = torch.sigmoid(arg)
    e = (6 + 5.25 * arg.abs()) * U
    inside, below = p >= 2.0 ** -126 * (1 + e), p < 2.0 ** -126 * (1 - e)
    assert bool(((y.double() - d * p).abs() <= (d * p).abs() * e)[inside].all())
    assert bool((y == 0)[below].all()) and int(below.sum()) > 100


def test_gates():
    """h = g * o without a residual, where x of ones is normalized to itself (eps 0)."""
    gate = torch.linspace(-120, 120, 24000).cuda().view(-1, 16)
    one = torch.ones(16, device="cuda")
    with torch.no_grad():
        h, _ = blocks.block_norms(torch.ones_like(gate), None, one, one, gate, sigmoid=True, eps=0.0)
    near(h, gate.double(), torch.ones_like(gate, dtype=torch.float64), 1)
