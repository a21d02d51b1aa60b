"""Kept activations and their gradients at both ends of a type: its lowest value, which masks
hold, and its largest, beyond the 127 * 2^121 that a code stands for at the largest exponent."""
import numpy as np
import pytest

import bit_microscaled_quantized_amd as nv
from tests import gpuio
from tests.test_gpu_blocks import held64, kept64, kept_buffers
from tests.test_gpu_norm import BF, F32, U, Tensors, f64, half_step

pytestmark = pytest.mark.gpu

MOST = 127 * 2.0 ** 121  # of the values that a code stands for


def ends(torch, t):
    """Magnitudes at and around 127 * 2^121 up to the type's largest."""
    top = torch.finfo(t).max
    a = torch.tensor([top, 127.5 * 2.0 ** 121, 127.25 * 2.0 ** 121, MOST, 126.5 * 2.0 ** 121, 126 * 2.0 ** 121,
                      64 * 2.0 ** 121], dtype=torch.float64).to(t)
    return torch.cat([a, -a])


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("cols,pad,off", [(32, 0, 0), (37, 3, 1), (5, 0, 0), (1, 2, 1)])
def test_codes_saturate_on_both_sides(dt, cols, pad, off):
    torch = gpuio.torch_cuda()
    v = ends(torch, torch.bfloat16 if dt == BF else torch.float32)
    rows = len(v)
    T = Tensors(rows, cols, dt, pad, off)
    # a row's value last, so that a ragged block's end has it, small ones before
    a = np.zeros((rows, cols))
    a[:, 0], a[:, -1] = 2.0 ** 121, v.double().numpy()
    x = T.put(a)
    x64 = f64(x)
    assert (x64 > MOST).sum() >= 2 and (x64 < -MOST).sum() >= 2
    g, codes, scales = kept_buffers(rows, cols)
    out = T.out()
    nv.nvfp4_gated_act(nv.NVFP4_ACT_NONE, x, None, dt, rows, cols, T.ld, 0, None, 0, codes, scales, None, None)
    nv.nvfp4_gated_act_backward(nv.NVFP4_ACT_NONE, codes, scales, None, None, None, dt, rows, cols, 0, None, 0, None, 0,
                                out, T.ld)
    T.check()
    g.check()
    q, s = kept64(x64)
    assert np.array_equal(codes.cpu().numpy(), q) and np.array_equal(scales.cpu().numpy(), s)
    assert np.array_equal(f64(out), held64(q, s))  # seven bits at an exponent of the type: exact
    assert np.abs(f64(out)).max() == MOST


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_the_layer_restores_finite_values(dtype):
    torch = gpuio.torch_cuda()
    from bit_microscaled_quantized_amd.blocks import keep8, restore8
    t = getattr(torch, dtype)
    for value, code in ((torch.finfo(t).min, -127), (torch.finfo(t).max, 127)):
        codes, scales = keep8(torch.full((2, 40), value, dtype=t, device="cuda"))
        assert bool((codes == code).all()) and bool((scales == 254).all())
        for out in (torch.bfloat16, torch.float32):
            assert bool((restore8(codes, scales, out).double() == code * 2.0 ** 121).all())


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("act,slopes", [(nv.NVFP4_ACT_SILU, (1.0, 0.0)), (nv.NVFP4_ACT_GELU, (1.0, 0.0)),
                                        (nv.NVFP4_ACT_NONE, (1.0, 1.0))])
def test_slopes_at_a_gates_ends(dt, act, slopes):
    """The activation is its argument, or 0, and its slope 1, or 0, exactly."""
    torch = gpuio.torch_cuda()
    t = torch.bfloat16 if dt == BF else torch.float32
    v = ends(torch, t).cuda()[:, None].repeat(1, 32)
    rows, cols = v.shape
    up = torch.full_like(v, 0.5)
    dy = torch.full_like(v, 2.0 ** -9)
    _, gc, gs = kept_buffers(rows, cols)
    _, uc, us = kept_buffers(rows, cols)
    y, again, dg, du = (torch.empty_like(v) for _ in range(4))
    nv.nvfp4_gated_act(act, v, up, dt, rows, cols, cols, cols, y, cols, gc, gs, uc, us)
    nv.nvfp4_gated_act_backward(act, gc, gs, uc, us, dy, dt, rows, cols, cols, dg, cols, du, cols, again, cols)
    kept = v.double().clamp(-MOST, MOST)
    kept = (kept / 2.0 ** 121).round() * 2.0 ** 121
    for out, at in ((y, v.double()), (again, kept)):
        want = torch.where(at > 0, at * slopes[0], at * slopes[1]) * 0.5
        assert torch.equal(out.double(), want)
    slope = torch.where(kept > 0, slopes[0], slopes[1]).double()
    assert torch.equal(dg.double(), slope * 0.5 * 2.0 ** -9)
    assert torch.equal(du.double(), kept * slope * 2.0 ** -9)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("act,slope", [(nv.NVFP4_ACT_SILU, 0.9276705118714867), (nv.NVFP4_ACT_GELU, 1.0829640838457826),
                                       (nv.NVFP4_ACT_RELU2, 2.0), (nv.NVFP4_ACT_NONE, 1.0)])
def test_gradients_at_an_ups_ends(dt, act, slope):
    """Beside a gate of 1: dy * up * slope, finite.  The slope is off by less than 30 u (p, the logistic function of at most
    1.7, by 5 + 4.25 * 1.7 u, as 1 - p is relative to p; factors of the other terms below 1.9), its product by two
    roundings more."""
    torch = gpuio.torch_cuda()
    t = torch.bfloat16 if dt == BF else torch.float32
    up = ends(torch, t).cuda()[:, None].repeat(1, 32)
    rows, cols = up.shape
    gate, dy = torch.ones_like(up), torch.full_like(up, 2.0 ** -9)
    _, gc, gs = kept_buffers(rows, cols)
    _, uc, us = kept_buffers(rows, cols)
    again, dg, du = (torch.empty_like(up) for _ in range(3))
    nv.nvfp4_gated_act(act, gate, up, dt, rows, cols, cols, cols, None, 0, gc, gs, uc, us)
    nv.nvfp4_gated_act_backward(act, gc, gs, uc, us, dy, dt, rows, cols, cols, dg, cols, du, cols, again, cols)
    want = ((up.double().clamp(-MOST, MOST) / 2.0 ** 121).round() * 2.0 ** 121) * (slope * 2.0 ** -9)
    assert bool(((dg.double() - want).abs() <= want.abs() * (half_step(dt) + 32 * U)).all())
    assert bool(torch.isfinite(again).all()) and bool(torch.isfinite(du).all())


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("act", ["silu", "gelu", "relu2"])
def test_masked_gates_have_no_gradient(dtype, act):
    """Gates that hold their type's lowest value beside others, in blocks of 32 of their own."""
    torch = gpuio.torch_cuda()
    from bit_microscaled_quantized_amd.blocks import gated_act
    t = getattr(torch, dtype)
    g = torch.Generator(device="cuda").manual_seed(4)
    gate = torch.randn(6, 96, generator=g, device="cuda").to(t)
    gate[:, 32:64] = torch.finfo(t).min
    gate.requires_grad_()
    up = torch.randn(6, 96, generator=g, device="cuda").to(t).requires_grad_()
    y = gated_act(gate, up, act)
    y.backward(torch.ones_like(y))
    assert bool((y[:, 32:64] == 0).all())
    for grad in (gate.grad, up.grad):
        assert bool(torch.isfinite(grad).all()) and bool((grad[:, 32:64] == 0).all())
        assert bool((grad[:, :32] != 0).any()) and bool((grad[:, 64:] != 0).any())
