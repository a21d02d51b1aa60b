"""Outputs in place of inputs of their own size, at widths where several waves share a row that ends
inside a vector, with more rows than a launch has workgroups: the results of the same calls with
tensors of their own, bit for bit."""
import pytest
import torch

import bit_microscaled_quantized_amd as nv

pytestmark = pytest.mark.gpu

BF, F32 = nv.NVFP4_BF16, nv.NVFP4_F32
# several waves a row, two rows and more a workgroup; one wave for several rows; whole vectors; read more than once
NORMS = [(BF, 700, 5119), (BF, 1300, 2051), (BF, 3000, 301), (BF, 9000, 61), (BF, 700, 5120), (BF, 600, 9001),
         (F32, 1200, 2049), (F32, 700, 8191), (F32, 3000, 130), (BF, 300, 41001)]


def tensors(dt, rows, cols, n):
    g = torch.Generator(device="cuda").manual_seed(rows + cols)
    t = torch.bfloat16 if dt == BF else torch.float32
    return [torch.randn(rows, cols, generator=g, device="cuda").to(t) for _ in range(n)], torch.randn(
        2, cols, generator=g, device="cuda").to(t)


def same(a, b):
    assert all(torch.equal(u, v) for u, v in zip(a, b))


@pytest.mark.parametrize("dt,rows,cols", NORMS)
@pytest.mark.parametrize("codes", [False, True])
def test_norms(dt, rows, cols, codes):
    (x, r, gate), (post, pre) = tensors(dt, rows, cols, 3)
    ld = (cols + 15) // 16 * 16

    def norms(x, r, h, y):
        stats = [torch.empty(rows, device="cuda") for _ in range(2)]
        q, s = torch.zeros(rows, ld, dtype=torch.int8, device="cuda"), torch.empty(rows, device="cuda")
        nv.nvfp4_block_norms(x, r, gate, dt, rows, cols, cols, cols, cols, 1, post, pre, dt, 1e-5, 0.5, h, cols,
                             None if codes else y, cols, q if codes else None, ld, s if codes else None, *stats)
        return [h.clone(), *stats] + ([q, s] if codes else [y.clone()])
    want = norms(x, r, torch.empty_like(x), torch.empty_like(x))
    for swap in (False, True):
        a, b = x.clone(), r.clone()
        same(norms(a, b, *((a, b) if swap else (b, a))), want)


@pytest.mark.parametrize("dt,rows,cols", NORMS)
@pytest.mark.parametrize("channel", [False, True])
def test_norms_backward(dt, rows, cols, channel):
    (dy, dh, h, x, gate), (post, pre) = tensors(dt, rows, cols, 5)
    if channel:
        gate = gate[0].clone()
    stats = [torch.rand(rows, device="cuda") + 0.5 for _ in range(2)]
    ws = torch.empty(nv.nvfp4_block_norms_backward_workspace_size(rows, cols), dtype=torch.uint8, device="cuda")

    def back(at, outs):
        """outs: names of the inputs that dx, dresidual and (a token's gate) dgate replace; None: none."""
        t = {k: v.clone() for k, v in at.items()}
        dx, dr, dg = (torch.empty_like(x) if n is None else t[n] for n in outs)
        if channel:
            dg = torch.empty(cols, device="cuda")
        sums = [torch.empty(cols, device="cuda") for _ in range(2)]
        nv.nvfp4_block_norms_backward(t["dy"], t["dh"], t["h"], t["x"], t["gate"], dt, rows, cols, cols, cols, cols, cols,
                                      0 if channel else cols, 1, post, pre, dt, *stats, 0.5, dx, cols, dr, cols, dg, cols,
                                      *sums, ws)
        return [dx, dr, dg, *sums]
    at = dict(dy=dy, dh=dh, h=h, x=x, gate=gate)
    want = back(at, (None, None, None))
    for outs in (("dy", "dh", "gate"), ("dh", "dy", "x"), ("x", "h", "dy"), ("h", "x", "dh")):
        same(back(at, outs), want)
    if not channel:
        same(back(at, ("gate", "dy", "h")), want)


@pytest.mark.parametrize("dt,rows,cols", [(BF, 700, 5119), (BF, 40, 37), (BF, 300, 5), (F32, 900, 2049), (F32, 70, 35),
                                          (F32, 90, 3), (BF, 64, 5120)])
@pytest.mark.parametrize("act", range(4))
def test_activation(dt, rows, cols, act):
    (gate, up, dy), _ = tensors(dt, rows, cols, 3)
    blocks = (cols + 31) // 32

    def forward(gate, up, y):
        kept = [torch.empty(rows, n, dtype=t, device="cuda") for _ in range(2) for n, t in ((cols, torch.int8),
                                                                                             (blocks, torch.uint8))]
        nv.nvfp4_gated_act(act, gate, up, dt, rows, cols, cols, cols, y, cols, *kept)
        return [y.clone(), *kept]
    want = forward(gate, up, torch.empty_like(gate))
    for k in range(2):
        a = [gate.clone(), up.clone()]
        same(forward(*a, a[k]), want)
    kept = want[1:]

    def backward(dy, at):
        outs = [torch.empty_like(gate) for _ in range(3)]
        if at is not None:
            outs[at] = dy
        nv.nvfp4_gated_act_backward(act, *kept, dy, dt, rows, cols, cols, *(v for o in outs for v in (o, cols)))
        return outs
    want = backward(dy.clone(), None)
    for at in range(3):
        same(backward(dy.clone(), at), want)
