"""The ways that dropout, the RMS norm and its backward pass take for wider and for more rows than
test_gpu_norm's: eight vectors a lane, FP32 rows of three, the accumulating rows of wide gradients,
and launches that stream past the caches, whose groups of lanes walk many rows.

Small ones repeat test_gpu_norm's checks; large ones compare with 64 bits on the device, by the same
counts of roundings."""
import pytest

import bit_microscaled_quantized_amd as nv
from tests import gpuio
from tests import test_gpu_norm as small
from tests.test_gpu_norm import BF, EPS, F32, SUM, U, Tensors, half_step

pytestmark = pytest.mark.gpu

# (dt, cols): three vectors a lane in FP32, eight in either type
WIDE = [(F32, 8193), (F32, 12288), (F32, 20481), (F32, 30001), (F32, 32768), (BF, 24576), (BF, 40961), (BF, 65536)]


@pytest.mark.parametrize("dt,cols", WIDE)
@pytest.mark.parametrize("mx", [False, True])
def test_rms_norm_of_wide_rows(dt, cols, mx):
    small.check_norm(3, cols, dt, 0.3, cols, small.run_norm(3, cols, dt, 3, 1, 0.3, cols, mx, BF))


@pytest.mark.parametrize("rows", [1, 5])
@pytest.mark.parametrize("dt,cols", WIDE)
def test_rms_norm_backward_of_wide_rows(rows, dt, cols):
    small.test_rms_norm_backward(rows, cols, dt, 3, 1, 0.3, F32)


@pytest.mark.parametrize("rows,cols,dt", [(300, 33001, F32), (259, 24601, BF), (600, 12001, F32), (520, 30001, F32)])
def test_rms_norm_backward_of_more_wide_rows_than_workgroups(rows, cols, dt):
    small.test_rms_norm_backward(rows, cols, dt, 0, 0, 0.0, F32)


def pcg(v):
    st = (v * 747796405 + 2891336453) & 0xFFFFFFFF
    w = (((st >> ((st >> 28) + 4)) ^ st) * 277803737) & 0xFFFFFFFF
    return (w >> 22) ^ w


def keep_scale(torch, rows, cols, p, seed):
    """small.keep_scale on the device."""
    key = pcg((seed & 0xFFFFFFFF) ^ pcg(seed >> 32))
    cut = int(round(p * 65536))
    i = torch.arange(rows * cols, device="cuda")
    w = pcg((i >> 1) ^ key)
    r16 = torch.where((i & 1) == 1, w >> 16, w & 0xFFFF)
    scale = float(torch.tensor(65536 / (65536 - cut)).float())
    return torch.where(r16 >= cut, scale, 0.0).double().view(rows, cols)


def test_keep_scale_is_the_host_form():
    torch = gpuio.torch_cuda()
    seed = 0x123456789ABCDEF0
    a, b = keep_scale(torch, 5, 33, 0.375, seed).cpu().numpy(), small.keep_scale(5, 33, 0.375, seed)
    assert (a == b).all() and (a == 0).any() and (a > 0).any()


def close(got, ref, tol, what):
    bad = ~((got.double() - ref).abs() <= tol)
    if bool(bad.any()):
        i = tuple(bad.nonzero()[0].tolist())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {i}: {float(got[i])} for "
                             f"{float(ref[i])} +- {float(tol.expand(ref.shape)[i])}")


class Large(Tensors):
    def __init__(self, rows, cols, dt, pad, off):
        super().__init__(rows, cols, dt, pad, off)
        self.rng = self.torch.Generator(device="cuda").manual_seed(rows + cols)

    def rand(self, std):
        v = self._view(self._buf())
        v.copy_(self.torch.randn(self.rows, self.cols, generator=self.rng, device="cuda") * std)
        return v


@pytest.mark.parametrize("rows,cols,dt,pad,off", [(4097, 8200, BF, 0, 0), (4097, 8201, BF, 3, 1), (2050, 8301, F32, 5, 3),
                                                  (70000, 500, BF, 4, 0)])
def test_dropout_past_the_caches(rows, cols, dt, pad, off):
    T = Large(rows, cols, dt, pad, off)
    x, y = T.rand(1.0), T.out()
    p, seed = 0.25, (9 << 32) | 5
    nv.nvfp4_dropout(x, dt, rows, cols, T.ld, p, seed, y, T.ld)
    T.check()
    ref = x.double() * keep_scale(T.torch, rows, cols, p, seed)
    close(y, ref, ref.abs() * (half_step(dt) + U), "y")


# launches of 128 MB and more; rows of one, two, three and five vectors a lane, of lanes inside a wave
MANY = [(4100, 5120, BF, 0, 0), (2050, 5119, F32, 5, 3), (1500, 16383, BF, 3, 1), (900, 24570, BF, 0, 0), (830, 12287, F32, 1, 1),
        (500, 20479, F32, 0, 0), (140000, 120, BF, 8, 0), (300000, 64, F32, 0, 0)]


@pytest.mark.parametrize("rows,cols,dt,pad,off", MANY)
@pytest.mark.parametrize("mx", [False, True])
def test_rms_norm_past_the_caches(rows, cols, dt, pad, off, mx):
    T = Large(rows, cols, dt, pad, off)
    torch = T.torch
    p, seed = 0.125, cols
    x, r = T.rand(1.0), T.rand(3.0)
    gamma = 1 + 0.2 * torch.randn(cols, generator=T.rng, device="cuda")
    h, rstd = T.out(), T.g.alloc((rows,), torch.float32)
    blocks = (cols + 31) // 32
    y = codes = scales = None
    if mx:
        codes, scales = T.g.alloc((rows, cols), torch.uint8), T.g.alloc((rows, blocks), torch.uint8)
    else:
        y = T.out()
    nv.nvfp4_rms_norm(x, r, dt, rows, cols, T.ld, T.ld, gamma, F32, EPS, p, seed, h, T.ld, y, T.ld, codes, scales, rstd)
    T.check()
    xk = x.double() * keep_scale(torch, rows, cols, p, seed)
    href = xk + r.double()
    dh = 2 * U * (xk.abs() + href.abs())
    del xk
    close(h, href, dh + half_step(dt) * href.abs(), "h")
    ms = href.square().mean(1) + EPS
    rref = ms.rsqrt()
    rel = ((2 * href.abs() * dh).mean(1) / ms + SUM + 3 * U) / 2 + 2 * U
    close(rstd, rref, rref * rel, "rstd")
    g = gamma.double()
    yref = href * rref[:, None] * g
    dy = yref.abs() * (rel[:, None] + 3 * U) + dh * rref[:, None] * g.abs()
    if not mx:
        close(y, yref, dy + half_step(dt) * yref.abs(), "y")
        return
    pad_cols = lambda t: torch.nn.functional.pad(t, (0, blocks * 32 - cols)).view(rows, blocks, 32)
    top, slack = pad_cols(yref).abs().amax(2), pad_cols(dy).amax(2)

    def exponent(a):  # smallest e with a <= 448 * 2^e
        m, e = torch.frexp(a)
        return torch.where(m <= 0.875, e - 9, e - 8).clamp(-127, 127)
    e = scales.int() - 127
    assert bool(((e >= exponent((top - slack).clamp(min=1e-300))) & (e <= exponent(top + slack))).all()), "block exponents"
    scale = torch.exp2(e.double()).repeat_interleave(32, 1)[:, :cols]
    tol = dy * (1 + 2.0 ** -4) + torch.maximum(yref.abs() * 2.0 ** -4, scale * 2.0 ** -10)
    close(codes.view(torch.float8_e4m3fn).float() * scale.float(), yref, tol, "codes")


# with the rows that a group of lanes adds to dgamma in turn, the groups of a workgroup, and the
# partial rows of a slice; 32 slices are added last
@pytest.mark.parametrize("rows,cols,dt,pad,off,adds", [
    (4100, 5120, BF, 0, 0, 9 + 1 + 16), (2050, 5119, F32, 5, 3, 5 + 1 + 16), (1500, 16383, BF, 3, 1, 6 + 1 + 8),
    (900, 24570, BF, 0, 0, 4 + 1 + 8), (830, 12287, F32, 1, 1, 4 + 1 + 8), (500, 20479, F32, 0, 0, 2 + 1 + 8),
    (20000, 2048, BF, 0, 0, 20 + 2 + 16), (140000, 120, BF, 8, 0, 9 + 32 + 16), (300000, 64, F32, 0, 0, 19 + 32 + 16)])
def test_rms_norm_backward_past_the_caches(rows, cols, dt, pad, off, adds):
    T = Large(rows, cols, dt, pad, off)
    torch = T.torch
    p, seed = 0.125, rows
    dy, dh, h = T.rand(1e-3), T.rand(2e-3), T.rand(3.0)
    gamma = 1 + 0.2 * torch.randn(cols, generator=T.rng, device="cuda")
    rstd = torch.rsqrt(h.double().square().mean(1) + EPS).float()
    dx, dr, dg = T.out(), T.out(), T.g.alloc((cols,), torch.float32, fill=float("nan"))
    n = nv.nvfp4_rms_norm_backward_workspace_size(rows, cols)
    ws = T.g.alloc((n // 4,), torch.float32, fill=float("nan"))
    nv.nvfp4_rms_norm_backward(dy, dh, h, dt, rows, cols, T.ld, T.ld, T.ld, gamma, F32, rstd, p, seed, dx, T.ld, dr, T.ld, dg,
                               ws)
    T.check()
    r = rstd.double()[:, None]
    n = h.double() * r
    gy = dy.double() * gamma.double()
    c = (gy * n).mean(1, keepdim=True)
    g = dh.double() + r * (gy - n * c)
    tol = (8 * U * (dh.double().abs() + r * (gy.abs() + (n * c).abs()))
           + r * n.abs() * (SUM + 4 * U) * (gy * n).abs().mean(1, keepdim=True))
    close(dr, g, tol + half_step(dt) * g.abs(), "dresidual")
    k = keep_scale(torch, rows, cols, p, seed)
    close(dx, g * k, k * tol + (half_step(dt) + U) * (g * k).abs(), "dx")
    # each term is a product of two roundings; then its additions, and those of the 32 slices
    terms = dy.double() * n
    close(dg, terms.sum(0), (adds + 32 + 3) * U * terms.abs().sum(0), "dgamma")
