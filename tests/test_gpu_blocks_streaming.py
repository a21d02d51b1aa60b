"""Calls of 128 MiB and more, whose loads and stores pass the caches by: the norms and their backward
pass with every gate against 64-bit computations, the activation and its backward pass against the
same rows in calls that do not (compared with 64 bits in test_gpu_blocks.py)."""
import pytest
import torch

import bit_microscaled_quantized_amd as nv
from tests import test_gpu_blocks as small

pytestmark = pytest.mark.gpu

BF, F32 = nv.NVFP4_BF16, nv.NVFP4_F32
STREAM = 128 << 20  # bytes


@pytest.mark.parametrize("rows,cols,dt,pad,off,kind", [(3280, 5119, BF, 3, 1, "token"), (1640, 5120, F32, 0, 0, "channel")])
def test_norms(rows, cols, dt, pad, off, kind):
    assert rows * cols * 4 * (2 if dt == BF else 4) >= STREAM
    small.test_norms(rows, cols, dt, pad, off, kind)


@pytest.mark.parametrize("rows,cols,dt,pad,off,kind", [
    (2190, 5119, BF, 3, 1, "token"), (2190, 5120, BF, 0, 0, "channel"), (1100, 5121, F32, 5, 3, "token"),
    (1100, 5120, F32, 0, 0, None), (690, 8191, F32, 0, 0, "channel")])
def test_norms_backward(rows, cols, dt, pad, off, kind):
    assert rows * cols * 6 * (2 if dt == BF else 4) >= STREAM
    small.test_norms_backward(rows, cols, dt, pad, off, kind)


@pytest.mark.parametrize("act", range(4))
@pytest.mark.parametrize("rows,cols,dt,gated", [(4500, 5119, BF, True), (1700, 20480, BF, False), (4400, 2560, F32, True),
                                                (3300, 5119, F32, False)])
def test_activation(rows, cols, dt, act, gated):
    size, part = (2 if dt == BF else 4), 300
    assert rows * cols * size * (3 if gated else 2) >= STREAM > part * cols * size * 4  # forward; backward has one more
    g = torch.Generator(device="cuda").manual_seed(rows + act)
    t = torch.bfloat16 if dt == BF else torch.float32
    gate, up, dy = (torch.randn(rows, cols, generator=g, device="cuda").to(t) for _ in range(3))
    if not gated:
        up = None

    def calls(gate, up, dy):
        n = gate.shape[0]
        kept = [torch.empty(n, w, dtype=k, device="cuda") for _ in range(2) for w, k in ((cols, torch.int8),
                                                                                          ((cols + 31) // 32, torch.uint8))]
        if up is None:
            kept[2:] = None, None
        y, again, dg, du = (torch.empty_like(gate) for _ in range(4))
        nv.nvfp4_gated_act(act, gate, up, dt, n, cols, cols, cols, y, cols, *kept)
        nv.nvfp4_gated_act_backward(act, *kept, dy, dt, n, cols, cols, dg, cols, None if up is None else du, cols, again, cols)
        return [y, *kept, dg, again] + ([] if up is None else [du])
    whole = calls(gate, up, dy)
    for first in range(0, rows, part):
        some = slice(first, min(first + part, rows))
        for a, b in zip(whole, calls(gate[some], None if up is None else up[some], dy[some])):
            assert a is b is None or torch.equal(a[some], b)
