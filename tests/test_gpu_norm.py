"""Dropout, the residual RMS norm (BF16 / FP32 / 8-bit output) and its backward
pass against plain 64-bit computations on the host.

Tolerances count roundings.  u = 2^-24 is half a step of FP32, half a step of
the output type eps / 2 (2^-8 for BF16, 2^-24 for FP32), of E4M3 2^-4 of a
normal value or 2^-10 of the block's scale.  A row sum is at most 64 additions
in a lane and 10 across lanes (wide rows: 8 in a vector, then one per vector of
the lane), so a sum of terms t is within 80 u sum |t|; a square root halves the
relative error of its argument."""
import numpy as np
import pytest

import bit_microscaled_quantized_amd as nv
from tests import gpuio

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
SUM = 80 * U
EPS = 1e-5


def _pcg(v):
    with np.errstate(over="ignore"):
        st = v * np.uint32(747796405) + np.uint32(2891336453)
        w = ((st >> ((st >> np.uint32(28)) + np.uint32(4))) ^ st) * np.uint32(277803737)
        return (w >> np.uint32(22)) ^ w


def keep_scale(rows, cols, p, seed):
    """Factor of each element: 0 where dropped, else 65536 / (65536 - cut)."""
    cut = int(round(float(np.float32(p)) * 65536))
    one = lambda v: _pcg(np.array([v & 0xFFFFFFFF], np.uint32))[0]
    key = one((seed & 0xFFFFFFFF) ^ int(one(seed >> 32)))
    i = np.arange(rows * cols, dtype=np.uint64)
    w = _pcg((i >> np.uint64(1)).astype(np.uint32) ^ key)
    r16 = np.where(i & np.uint64(1), w >> np.uint32(16), w & np.uint32(0xFFFF))
    return np.where(r16 >= cut, float(np.float32(65536 / (65536 - cut))), 0.0).reshape(rows, cols)


def test_keep_bits_are_the_sr_bits(ora):
    seed = 0x123456789ABCDEF0
    got = keep_scale(3, 7, 0.5, seed).ravel() > 0
    assert list(got) == [ora.sr_bits(seed, i) >= 32768 for i in range(21)]


class Tensors:
    """Device tensors of one call: inputs as slices of wider buffers (`pad`
    columns after each row, `off` elements before the first), outputs between
    guard zones with the same layout and the gaps checked."""

    def __init__(self, rows, cols, dt, pad, off):
        self.torch = gpuio.torch_cuda()
        self.rows, self.cols, self.ld, self.off = rows, cols, cols + pad, off
        self.t = self.torch.bfloat16 if dt == nv.NVFP4_BF16 else self.torch.float32
        self.g = gpuio.Guarded()
        self.gaps = []

    def _buf(self):
        return self.g.alloc((max(self.rows * self.ld + self.off, 1),), self.t, fill=7.0)

    def _view(self, b):
        return b[self.off:self.off + self.rows * self.ld].view(self.rows, self.ld)[:, :self.cols]

    def put(self, a):
        b = self._buf()
        v = self._view(b)
        v.copy_(self.torch.from_numpy(np.ascontiguousarray(a, np.float32)).cuda())
        return v

    def out(self):
        b = self._buf()
        self.gaps.append(b)
        return self._view(b)

    def check(self):
        self.torch.cuda.synchronize()
        self.g.check()
        for b in self.gaps:
            c = b.clone()
            self._view(c).fill_(7.0)
            assert bool((c == 7.0).all()), "a gap between rows was written"


def f64(t):
    return t.double().cpu().numpy()


def half_step(dt):
    return 2.0 ** -8 if dt == nv.NVFP4_BF16 else U


def data(rng, rows, cols, std=1.0):
    a = rng.normal(0, std, (rows, cols))
    a[:, rng.integers(cols)] *= 10
    return a


def close(got, ref, tol, what):
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.size} off, first at {np.argwhere(bad)[0]}: "
                           f"{got[bad][0]} for {ref[bad][0]} +- {np.broadcast_to(tol, ref.shape)[bad][0]}")


BF, F32 = nv.NVFP4_BF16, nv.NVFP4_F32
SHAPES = [(0, 8), (1, 1), (1, 2), (5, 1), (3, 7), (2, 31), (33, 32), (17, 33), (9, 64), (40, 127), (7, 128),
          (65, 129), (5, 255), (16, 513), (4, 1024), (3, 2049), (130, 5120), (9, 5119), (2, 12289), (2, 20479),
          (3, 32769), (2, 70001)]


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("dt,pad,off", [(BF, 0, 0), (BF, 3, 1), (BF, 64, 0), (F32, 0, 0), (F32, 5, 3)])
def test_dropout(rows, cols, dt, pad, off):
    rng = np.random.default_rng(rows * 31 + cols)
    for p, seed in ((0.25, 5), (0.0, 1), (0.999, (7 << 32) | 3)):
        T = Tensors(rows, cols, dt, pad, off)
        x, y = T.put(data(rng, rows, cols)), T.out()
        nv.nvfp4_dropout(x, dt, rows, cols, T.ld, p, seed, y, T.ld)
        T.check()
        ref = f64(x) * keep_scale(rows, cols, p, seed)
        close(f64(y), ref, np.abs(ref) * (half_step(dt) + U), f"p {p}")


def test_dropout_drops_what_is_not_a_number_and_its_share():
    torch = gpuio.torch_cuda()
    rows, cols, p, seed = 64, 1024, 0.3, 77
    kept = keep_scale(rows, cols, p, seed) > 0
    x = torch.full((rows, cols), float("inf"), device="cuda")
    x[::2] = float("nan")
    nv.nvfp4_dropout(x, F32, rows, cols, cols, p, seed, x, cols)  # in place
    got = x.cpu().numpy()
    assert (got[~kept] == 0).all() and np.isinf(got[1::2][kept[1::2]]).all() and np.isnan(got[::2][kept[::2]]).all()
    assert abs((~kept).mean() - p) < 5 * np.sqrt(p * (1 - p) / kept.size)


def norm_ref(x, r, gamma, p, seed):
    k = keep_scale(*x.shape, p, seed)
    h = x * k + r
    rstd = 1 / np.sqrt((h * h).mean(1) + EPS)
    return k, h, rstd, h * rstd[:, None] * gamma


def run_norm(rows, cols, dt, pad, off, p, seed, mx, gdt, with_residual=True, rng=None):
    rng = rng or np.random.default_rng(rows * 17 + cols)
    T = Tensors(rows, cols, dt, pad, off)
    torch = T.torch
    x = T.put(data(rng, rows, cols))
    r = T.put(data(rng, rows, cols, 3.0)) if with_residual else None
    gamma = torch.from_numpy(1 + 0.2 * rng.normal(0, 1, cols)).cuda().to(torch.bfloat16 if gdt == BF else torch.float32)
    h, rstd = T.out(), T.g.alloc((rows,), torch.float32)
    y = codes = scales = None
    blocks = (cols + 31) // 32
    if mx:
        codes, scales = T.g.alloc((rows, cols), torch.uint8), T.g.alloc((rows, blocks), torch.uint8)
    else:
        y = T.out()
    nv.nvfp4_rms_norm(x, r, dt, rows, cols, T.ld, T.ld, gamma, gdt, EPS, p, seed, h, T.ld, y, T.ld, codes, scales,
                      rstd)
    T.check()
    return x, r, gamma, h, rstd, y, codes, scales


def check_norm(rows, cols, dt, p, seed, out):
    x, r, gamma, h, rstd, y, codes, scales = out
    xs, g = f64(x), f64(gamma)
    rs = f64(r) if r is not None else np.zeros_like(xs)
    k, href, rref, yref = norm_ref(xs, rs, g, p, seed)
    dh = 2 * U * (np.abs(xs * k) + np.abs(href))       # the product and the sum that form h
    close(f64(h), href, dh + half_step(dt) * np.abs(href), "h")
    # mean(h^2): its terms' errors, the sum's, the division and the addition; then root and quotient
    ms = 1 / rref ** 2
    rel = ((2 * np.abs(href) * dh).mean(1) / ms + SUM + 3 * U) / 2 + 2 * U
    close(f64(rstd), rref, rref * rel, "rstd")
    dy = np.abs(yref) * (rel[:, None] + 3 * U) + dh * rref[:, None] * np.abs(g)
    if y is not None:
        close(f64(y), yref, dy + half_step(dt) * np.abs(yref), "y")
        return
    blocks = scales.shape[1] if rows else 0
    if not rows:
        return
    pad = blocks * 32 - cols
    yb = np.pad(yref, ((0, 0), (0, pad))).reshape(rows, blocks, 32)
    db = np.pad(dy, ((0, 0), (0, pad))).reshape(rows, blocks, 32)
    top, slack = np.abs(yb).max(2), db.max(2)

    def exponent(a):  # smallest e with a <= 448 * 2^e
        m, e = np.frexp(a)
        return np.where(a <= 0, -127, np.clip(np.where(m <= 0.875, e - 9, e - 8), -127, 127))
    e = scales.cpu().numpy().astype(int) - 127
    assert ((e >= exponent(top - slack)) & (e <= exponent(top + slack))).all(), "block exponents"
    torch = gpuio.torch_cuda()
    val = codes.view(torch.float8_e4m3fn).float().double().cpu().numpy()
    scale = np.repeat(np.exp2(e.astype(float)), 32, 1)[:, :cols]
    tol = dy * (1 + 2.0 ** -4) + np.maximum(np.abs(yref) * 2.0 ** -4, scale * 2.0 ** -10)
    close(val * scale, yref, tol, "codes")


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("dt,pad,off,p,gdt", [(BF, 0, 0, 0.1, BF), (BF, 3, 1, 0.0, F32), (F32, 0, 0, 0.5, F32),
                                              (F32, 5, 3, 0.0, BF)])
@pytest.mark.parametrize("mx", [False, True])
def test_rms_norm(rows, cols, dt, pad, off, p, gdt, mx):
    seed = (cols << 33) | rows
    check_norm(rows, cols, dt, p, seed, run_norm(rows, cols, dt, pad, off, p, seed, mx, gdt))


@pytest.mark.parametrize("mx", [False, True])
def test_rms_norm_without_residual(mx):
    check_norm(5, 333, BF, 0.2, 9, run_norm(5, 333, BF, 1, 1, 0.2, 9, mx, BF, with_residual=False))


def test_rms_norm_in_place_and_without_saved_outputs():
    torch = gpuio.torch_cuda()
    rows, cols = 6, 5121
    _, _, _, h, _, y, _, _ = run_norm(rows, cols, BF, 0, 0, 0.1, 3, False, BF)
    x, r, gamma, *_ = run_norm(rows, cols, BF, 0, 0, 0.1, 3, False, BF)
    only = torch.empty_like(y)
    nv.nvfp4_rms_norm(x, r, BF, rows, cols, cols, cols, gamma, BF, EPS, 0.1, 3, None, 0, only, cols, None, None, None)
    nv.nvfp4_rms_norm(x, r, BF, rows, cols, cols, cols, gamma, BF, EPS, 0.1, 3, r, cols, x, cols, None, None, None)
    torch.cuda.synchronize()
    assert torch.equal(only, y) and torch.equal(r, h) and torch.equal(x, y)


def test_rms_norm_special_values():
    """An all-zero row, infinities and NaN: zero codes under the smallest scale, and
    NaN blocks exactly where the row holds what is not finite."""
    torch = gpuio.torch_cuda()
    x = torch.randn(5, 96, device="cuda")
    x[0] = 0
    x[1, 40] = float("inf")
    x[2, 5] = float("nan")
    x[3] *= 1e-30
    gamma = torch.ones(96, device="cuda")
    y, rstd = torch.empty_like(x), torch.empty(5, device="cuda")
    codes = torch.empty(5, 96, dtype=torch.uint8, device="cuda")
    scales = torch.empty(5, 3, dtype=torch.uint8, device="cuda")
    common = (x, None, F32, 5, 96, 96, 96, gamma, F32)
    nv.nvfp4_rms_norm(*common, EPS, 0.0, 0, None, 0, y, 96, None, None, rstd)
    nv.nvfp4_rms_norm(*common, EPS, 0.0, 0, None, 0, None, 0, codes, scales, None)
    yc, c, s = y.cpu().numpy(), codes.cpu().numpy(), scales.cpu().numpy()
    assert (yc[0] == 0).all() and (c[0] == 0).all() and (s[0] == 0).all()
    assert rstd[1] == 0 and (np.delete(yc[1], 40) == 0).all() and np.isnan(yc[1, 40])  # 0 * inf
    assert list(s[1]) == [0, 255, 0] and (c[1, 32:64] == 0x7F).all()
    assert np.isnan(yc[2]).all() and (s[2] == 255).all()
    assert np.isfinite(yc[3:]).all() and (s[3:] < 255).all()


def back_ref(dy, dh, h, gamma, rstd, k):
    n = h * rstd[:, None]
    gy = dy * gamma
    c = (gy * n).mean(1, keepdims=True)
    g = dh + rstd[:, None] * (gy - n * c)
    tol = (8 * U * (np.abs(dh) + rstd[:, None] * (np.abs(gy) + np.abs(n * c)))
           + rstd[:, None] * np.abs(n) * (SUM + 4 * U) * np.abs(gy * n).mean(1, keepdims=True))
    return g, g * k, (dy * n).sum(0), tol, n


@pytest.mark.parametrize("rows,cols", SHAPES + [(1500, 96), (1025, 300), (700, 2050)])
@pytest.mark.parametrize("dt,pad,off,p,gdt", [(BF, 0, 0, 0.1, BF), (BF, 3, 1, 0.0, F32), (F32, 0, 0, 0.5, F32),
                                              (F32, 5, 3, 0.0, BF)])
def test_rms_norm_backward(rows, cols, dt, pad, off, p, gdt):
    rng = np.random.default_rng(rows * 13 + cols)
    seed = 11 + rows
    T = Tensors(rows, cols, dt, pad, off)
    torch = T.torch
    dy, dh, h = (T.put(data(rng, rows, cols, s)) for s in (1e-3, 2e-3, 3.0))
    gamma = torch.from_numpy(1 + 0.2 * rng.normal(0, 1, cols)).cuda().to(torch.bfloat16 if gdt == BF else torch.float32)
    rstd = torch.rsqrt(h.double().square().mean(1) + EPS).float()
    dx, dr, dg = T.out(), T.out(), T.g.alloc((cols,), torch.float32, fill=float("nan"))
    ws = T.g.alloc((nv.nvfp4_rms_norm_backward_workspace_size(rows, cols) // 4,), torch.float32, fill=float("nan"))
    nv.nvfp4_rms_norm_backward(dy, dh, h, dt, rows, cols, T.ld, T.ld, T.ld, gamma, gdt, rstd, p, seed, dx, T.ld, dr,
                               T.ld, dg, ws)
    T.check()
    k = keep_scale(rows, cols, p, seed)
    g, gx, dgr, tol, n = back_ref(f64(dy), f64(dh), f64(h), f64(gamma), f64(rstd), k)
    close(f64(dr), g, tol + half_step(dt) * np.abs(g), "dresidual")
    close(f64(dx), gx, k * tol + (half_step(dt) + U) * np.abs(gx), "dx")
    # a column: rows of a workgroup, its groups of rows, the partial sums (at most 64 in a slice, then 8)
    adds = rows / 512 + 16 + 64 + 8 + 4
    close(f64(dg), dgr, adds * U * (np.abs(f64(dy) * n)).sum(0), "dgamma")


@pytest.mark.parametrize("cols", [96, 5000, 40000])
def test_rms_norm_backward_parts(cols):
    """Each output alone, without dh, and over dy in place: the values of the whole call."""
    torch = gpuio.torch_cuda()
    rng = np.random.default_rng(cols)
    rows = 7
    T = Tensors(rows, cols, F32, 0, 0)
    dy, h = T.put(data(rng, rows, cols, 1e-3)), T.put(data(rng, rows, cols))
    gamma = torch.ones(cols, device="cuda")
    rstd = torch.rsqrt(h.square().mean(1) + EPS)
    ws = torch.empty(nv.nvfp4_rms_norm_backward_workspace_size(rows, cols), dtype=torch.uint8, device="cuda")

    def call(dx, dr, dg, dy=dy, ws=ws):
        nv.nvfp4_rms_norm_backward(dy, None, h, F32, rows, cols, cols, 0, cols, gamma, F32, rstd, 0.25, 4, dx, cols,
                                   dr, cols, dg, ws)
    dx, dr, dg = torch.empty_like(h), torch.empty_like(h), torch.empty_like(gamma)
    call(dx, dr, dg)
    a, b, c, d = torch.empty_like(h), torch.empty_like(h), torch.empty_like(gamma), dy.clone()
    call(a, None, None, ws=None)
    call(None, b, None, ws=None)
    call(None, None, c)
    call(None, d, None, dy=d, ws=None)
    torch.cuda.synchronize()
    assert torch.equal(a, dx) and torch.equal(b, dr) and torch.equal(c, dg) and torch.equal(d, dr)


@pytest.mark.parametrize("rows,cols,p", [(3, 40, 0.0), (4, 257, 0.3)])
def test_rms_norm_backward_against_differences(rows, cols, p):
    """<gradient, direction> against the central difference of <y, dy> + <h, dh> in 64 bits."""
    torch = gpuio.torch_cuda()
    rng = np.random.default_rng(5)
    x, r, dy, dh, ex, er = (rng.normal(0, 1, (rows, cols)) for _ in range(6))
    gamma, eg = 1 + 0.2 * rng.normal(0, 1, cols), rng.normal(0, 1, cols)
    dev = lambda a: torch.from_numpy(a).float().cuda()
    seed = 21
    h, y, rstd = torch.empty(rows, cols, device="cuda"), torch.empty(rows, cols, device="cuda"), \
        torch.empty(rows, device="cuda")
    nv.nvfp4_rms_norm(dev(x), dev(r), F32, rows, cols, cols, cols, dev(gamma), F32, EPS, p, seed, h, cols, y, cols,
                      None, None, rstd)
    dx, dr, dg = torch.empty_like(h), torch.empty_like(h), torch.empty(cols, device="cuda")
    ws = torch.empty(nv.nvfp4_rms_norm_backward_workspace_size(rows, cols), dtype=torch.uint8, device="cuda")
    nv.nvfp4_rms_norm_backward(dev(dy), dev(dh), h, F32, rows, cols, cols, cols, cols, dev(gamma), F32, rstd, p, seed,
                               dx, cols, dr, cols, dg, ws)

    def value(s):
        _, hh, _, yy = norm_ref(x + s * ex, r + s * er, gamma + s * eg, p, seed)
        return (yy * dy).sum() + (hh * dh).sum()
    e = 1e-4
    diff = (value(e) - value(-e)) / (2 * e)
    parts = (f64(dx) * ex, f64(dr) * er, f64(dg) * eg)
    got = sum(q.sum() for q in parts)
    size = sum(np.abs(q).sum() for q in parts)
    # FP32 rounding of inputs, saved h and sums; e^2 times the third derivative, of order one per term
    assert abs(got - diff) <= size * (SUM + 20 * U + 10 * e * e)
