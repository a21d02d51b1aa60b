"""The norms around a block with its gate and residual scale, the gated activation
whose inputs are kept in 8 bits, and their backward passes against plain 64-bit
computations on the host.

Tolerances count roundings, as in test_gpu_norm.py: u = 2^-24, SUM = 80 u for a row's
sum relative to its terms' magnitudes.  The logistic function of v has a relative error
of (1.25 |v| (1 - p) + 5) u: the exponent's product by |v|, the instructions' 1 ulp
each (2 u), the sum's.  A sum over the rows takes one rounding a row and fewer than 64
more for its partial sums.  Codes and scale bytes of kept inputs are exact."""
import numpy as np
import pytest

import bit_microscaled_quantized_amd as nv
from tests import gpuio
from tests.test_gpu_int8 import act64, check_pads, code_buffers
from tests.test_gpu_norm import EPS, F32, BF, SUM, U, Tensors, close, data, f64, half_step

pytestmark = pytest.mark.gpu

SHAPES = [(0, 8), (1, 1), (1, 2), (5, 1), (3, 7), (2, 31), (33, 32), (17, 33), (9, 64), (40, 127), (7, 128),
          (65, 129), (5, 255), (16, 513), (1030, 1025), (3, 2049), (130, 5120), (9, 5119), (2, 12289), (2, 20479),
          (3, 32769), (2, 70001)]
KINDS = [(BF, 0, 0), (BF, 3, 1), (F32, 0, 0), (F32, 5, 3)]
GATES = [None, "token", "channel"]


def logistic(v):
    """(p, 1 - p, relative error of p in u)"""
    with np.errstate(over="ignore"):
        p, q = 1 / (1 + np.exp(-v)), 1 / (1 + np.exp(v))
    return p, q, 1.25 * np.abs(v) * q + 5


def gate64(gate, sigmoid):
    """Factor, its slope, and the relative errors of both in u."""
    if gate is None:
        return 1.0, 0.0, 0.0, 0.0
    if not sigmoid:
        return gate, np.ones_like(gate), 0.0, 0.0
    p, q, e = logistic(gate)
    # 1 - p: p's error and a rounding of at most p's size, over q
    return p, p * q, e, e + (p * e + 2) / np.maximum(q, 1e-30) + 1


class Gate:
    """A gate of a call: per token, one row for all (also as a slice of a wider buffer), or none."""

    def __init__(self, T, rng, rows, cols, kind):
        self.kind, self.t, self.ld = kind, None, 0
        if kind == "token":
            self.t, self.ld = T.put(rng.normal(0, 1.5, (rows, cols))), T.ld
        elif kind == "channel":
            one = Tensors(1, cols, BF if T.t == T.torch.bfloat16 else F32, 0, T.off)
            self.t = one.put(rng.normal(0.5, 0.3, (1, cols)))

    def f64(self):
        return None if self.t is None else f64(self.t)


def forward64(x, res, gate, sigmoid, post, pre, scale):
    """h, y, both rstd, and the error bounds of h and y before their rounding to the output's type."""
    r1 = 1 / np.sqrt((x * x).mean(1, keepdims=True) + EPS)
    g, _, eg, _ = gate64(gate, sigmoid)
    o = scale * g * (x * r1 * post)
    h = res + o
    eh = np.abs(o) * (SUM / 2 + (8 + eg) * U) + np.abs(h) * U
    ms = (h * h).mean(1, keepdims=True) + EPS
    r2 = 1 / np.sqrt(ms)
    rel = SUM / 2 + 4 * U + (np.abs(h) * eh).mean(1, keepdims=True) / ms
    y = h * r2 * pre
    ey = np.abs(y) * (rel + 3 * U) + eh * np.abs(r2 * pre)
    return h, y, r1[:, 0], r2[:, 0], eh, ey, rel[:, 0]


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("dt,pad,off", KINDS)
@pytest.mark.parametrize("kind", GATES)
def test_norms(rows, cols, dt, pad, off, kind):
    rng = np.random.default_rng(rows * 31 + cols)
    torch = gpuio.torch_cuda()
    T = Tensors(rows, cols, dt, pad, off)
    x, r = T.put(data(rng, rows, cols)), T.put(data(rng, rows, cols, 3.0))
    G = Gate(T, rng, rows, cols, kind)
    gdt = F32 if pad else dt
    post, pre = (torch.from_numpy(rng.normal(1, 0.2, cols)).to(torch.float32 if gdt == F32 else T.t).cuda()
                 for _ in range(2))
    for sigmoid, residual, codes_out in ((1, True, False), (0, False, False), (1, True, True)):
        h, y = T.out(), T.out()
        r1, r2 = (T.g.alloc((max(rows, 1),), torch.float32) for _ in range(2))
        cg, codes, scales = code_buffers(rows, cols, 16)
        nv.nvfp4_block_norms(x, r if residual else None, G.t, dt, rows, cols, T.ld, T.ld, G.ld, sigmoid, post, pre, gdt,
                             EPS, 0.75, h, T.ld, None if codes_out else y, T.ld, codes if codes_out else None,
                             codes.stride(0), scales if codes_out else None, r1, r2)
        T.check()
        h64, y64, r164, r264, eh, ey, rel = forward64(f64(x), f64(r) if residual else 0.0 * f64(x), G.f64(), sigmoid,
                                                      f64(post), f64(pre), 0.75)
        hs = half_step(dt)
        close(f64(h), h64, eh + (np.abs(h64) + eh) * hs + 2.0 ** -140, "h")
        close(f64(r1)[:rows], r164, r164 * (SUM / 2 + 4 * U), "post_rstd")
        close(f64(r2)[:rows], r264, r264 * rel, "pre_rstd")
        if not codes_out:
            close(f64(y), y64, ey + (np.abs(y64) + ey) * hs + 2.0 ** -140, "y")
            continue
        if rows == 0:
            continue
        top, worst = np.abs(y64).max(1), (np.abs(y64) + ey).max(1)
        c = check_pads(cg, codes, rows, cols).astype(np.float64)
        s = scales.cpu().numpy().astype(np.float64)
        assert (np.abs(s - top / 127) <= (worst - top) / 127 + 2 * U * top / 127).all()
        step = np.maximum(top / 127, 1e-300)[:, None]
        offby = ey / step + 127 * ((worst - top) / np.maximum(top, 1e-300))[:, None] + 127 * 3 * U
        assert (np.abs(c - y64 / step) <= 0.5 + offby).all()


def rows_sum(rows):
    return (rows + 64) * U


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("dt,pad,off", KINDS)
@pytest.mark.parametrize("kind", GATES)
def test_norms_backward(rows, cols, dt, pad, off, kind):
    rng = np.random.default_rng(rows * 17 + cols)
    torch = gpuio.torch_cuda()
    T = Tensors(rows, cols, dt, pad, off)
    x, h = T.put(data(rng, rows, cols)), T.put(data(rng, rows, cols, 3.0))
    dy, dh = T.put(data(rng, rows, cols)), T.put(data(rng, rows, cols))
    G = Gate(T, rng, rows, cols, kind)
    gdt = F32 if pad else dt
    post, pre = (torch.from_numpy(rng.normal(1, 0.2, cols)).to(torch.float32 if gdt == F32 else T.t).cuda()
                 for _ in range(2))
    X, H, DY = f64(x), f64(h), f64(dy)
    r1t, r2t = (torch.from_numpy(1 / np.sqrt((v * v).mean(1) + EPS)).float().cuda() for v in (X, H))
    R1, R2 = f64(r1t)[:, None], f64(r2t)[:, None]
    size = nv.nvfp4_block_norms_backward_workspace_size(rows, cols)
    ws = T.g.alloc((size + 4,), torch.uint8)
    hs = half_step(dt)
    for sigmoid, with_dh, some in ((1, True, None), (0, False, None), (1, True, "dx"), (0, True, "dpost")):
        dx, dr = T.out(), T.out()
        dg = T.out() if kind != "channel" else T.g.alloc((cols,), torch.float32)
        dpost, dpre = (T.g.alloc((cols,), torch.float32) for _ in range(2))
        pick = lambda name, t: t if some in (None, name) else None  # noqa: E731
        nv.nvfp4_block_norms_backward(
            dy, dh if with_dh else None, h, x, G.t, dt, rows, cols, T.ld, T.ld, T.ld, T.ld, G.ld, sigmoid, post, pre, gdt,
            r1t, r2t, 0.75, pick("dx", dx), T.ld, pick("dr", dr), T.ld, pick("dg", dg) if kind else None, T.ld,
            pick("dpost", dpost), pick("dpre", dpre), ws, size)
        T.check()
        pr, po = f64(pre), f64(post)
        n, a = H * R2, DY * pr
        mean = (a * n).mean(1, keepdims=True) if rows else 0.0 * R1
        abs_mean = np.abs(a * n).mean(1, keepdims=True) if rows else 0.0 * R1
        t = (f64(dh) if with_dh else 0.0) + R2 * (a - n * mean)
        et = (np.abs(R2) * (np.abs(a) * 3 * U + np.abs(n) * (SUM * abs_mean + 5 * U * np.abs(mean))) + 2 * U * np.abs(t))
        g, slope, eg, es = gate64(G.f64(), sigmoid)
        m = X * R1
        d = 0.75 * t * g
        ed = 0.75 * np.abs(g) * et + np.abs(d) * (3 + eg) * U
        b, eb = d * po, ed * np.abs(po) + np.abs(d * po) * U
        mean_b = (b * m).mean(1, keepdims=True) if rows else 0.0 * R1
        abs_b = np.abs(b * m).mean(1, keepdims=True) if rows else 0.0 * R1
        err_b = (eb * np.abs(m)).mean(1, keepdims=True) if rows else 0.0 * R1
        ref = R1 * (b - m * mean_b)
        ex = R1 * (eb + np.abs(m) * (err_b + SUM * abs_b + 5 * U * np.abs(mean_b))) + 2 * U * np.abs(ref)
        tiny = 2.0 ** -140
        if some in (None, "dx"):
            close(f64(dx), ref, ex + (np.abs(ref) + ex) * hs + tiny, "dx")
        if some in (None, "dr"):
            close(f64(dr), t, et + (np.abs(t) + et) * hs + tiny, "dresidual")
        if some is None:
            close(f64(dpre), (DY * n).sum(0), np.abs(DY * n).sum(0) * (rows_sum(rows) + 2 * U), "dpre_gamma")
        if some in (None, "dpost"):
            close(f64(dpost), (d * m).sum(0), (ed * np.abs(m)).sum(0) + np.abs(d * m).sum(0) * (rows_sum(rows) + 4 * U),
                  "dpost_gamma")
        if some is None and kind:
            term = 0.75 * t * m * po * slope
            eterm = 0.75 * et * np.abs(m * po * slope) + np.abs(term) * (6 + es) * U
            if kind == "token":
                close(f64(dg), term, eterm + (np.abs(term) + eterm) * hs + tiny, "dgate")
            else:
                close(f64(dg), term.sum(0), eterm.sum(0) + np.abs(term).sum(0) * rows_sum(rows), "dgate")


def kept64(v):
    """Codes and bytes of kept values by their definition."""
    rows, cols = v.shape
    blocks = (cols + 31) // 32
    p = np.zeros((rows, blocks * 32))
    p[:, :cols] = v
    p = p.reshape(rows, blocks, 32)
    top = np.abs(p).max(2)
    with np.errstate(divide="ignore"):
        e = np.ceil(np.log2(top / 127))
    e = np.where(top > 127 * 2.0 ** e, e + 1, e)
    e = np.where(top <= 127 * 2.0 ** (e - 1), e - 1, e)
    e = np.clip(e, -133, 121)
    q = np.clip(np.rint(p / 2.0 ** e[..., None]), -127, 127)
    return q.reshape(rows, -1)[:, :cols], e + 133


def held64(codes, scales):
    return codes.astype(np.float64) * 2.0 ** (np.repeat(scales.astype(np.float64), 32, 1)[:, :codes.shape[1]] - 133)


def kept_buffers(rows, cols):
    torch = gpuio.torch_cuda()
    g = gpuio.Guarded()
    # one byte past the guard zone's alignment: codes may lie anywhere
    codes = g.alloc((rows * cols + 1,), torch.int8)[1:].view(rows, cols)
    return g, codes, g.alloc((rows, (cols + 31) // 32), torch.uint8)


def inputs(rng, rows, cols):
    a = data(rng, rows, cols)
    if rows > 2:  # powers of two apart from block to block, down to nothing
        a[1] *= 2.0 ** rng.integers(-40, 40, cols // 32 + 1).repeat(32)[:cols]
        a[2, ::2] = 0.0
    return a


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("dt,pad,off", KINDS)
def test_activation_and_its_backward(rows, cols, dt, pad, off):
    rng = np.random.default_rng(rows * 13 + cols)
    T = Tensors(rows, cols, dt, pad, off)
    gate, up, dy = T.put(inputs(rng, rows, cols)), T.put(inputs(rng, rows, cols)), T.put(data(rng, rows, cols))
    hs = half_step(dt)
    for act in range(4):
        for gated in (False, True):
            kg, gc, gs = kept_buffers(rows, cols)
            ku, uc, us = kept_buffers(rows, cols)
            y, again, dg, du = T.out(), T.out(), T.out(), T.out()
            nv.nvfp4_gated_act(act, gate, up if gated else None, dt, rows, cols, T.ld, T.ld, y, T.ld, gc, gs,
                               uc if gated else None, us if gated else None)
            nv.nvfp4_gated_act_backward(act, gc, gs, uc if gated else None, us if gated else None, dy, dt, rows, cols,
                                        T.ld, dg, T.ld, du if gated else None, T.ld, again, T.ld)
            T.check()
            kg.check()
            ku.check()
            if rows == 0:
                continue
            a, rel = act64(act, f64(gate))
            ref = a * (f64(up) if gated else 1.0)
            # where the logistic function is below 2^-126 it may come out as 0
            floor = 2.0 ** -120 * np.maximum(np.abs(f64(gate) * (f64(up) if gated else 1.0)), 1.0)
            close(f64(y), ref, np.abs(ref) * (hs + (rel + 1) * U) + floor, f"y of {act}")
            for t, c, s in ((gate, gc, gs), (up, uc, us))[:1 + gated]:
                q, e = kept64(f64(t))
                assert np.array_equal(c.cpu().numpy(), q) and np.array_equal(s.cpu().numpy(), e)
            v = held64(gc.cpu().numpy(), gs.cpu().numpy())
            u = held64(uc.cpu().numpy(), us.cpu().numpy()) if gated else np.ones_like(v)
            a, rel = act64(act, v)
            floor = 2.0 ** -120 * np.maximum(np.abs(v * u), 1.0)
            close(f64(again), a * u, np.abs(a * u) * (hs + (rel + 1) * U) + floor, f"y again of {act}")
            if gated:
                close(f64(du), f64(dy) * a, np.abs(f64(dy) * a) * (hs + (rel + 1) * U) + floor * np.abs(f64(dy)),
                      f"dup of {act}")
            if act in (nv.NVFP4_ACT_SILU, nv.NVFP4_ACT_GELU):
                gelu = act == nv.NVFP4_ACT_GELU
                C = np.sqrt(8 / np.pi)
                arg = C * (v + 0.044715 * v ** 3) if gelu else v
                D = C * (1 + 3 * 0.044715 * v * v) if gelu else 1.0
                p, q, _ = logistic(arg)
                e = (4.25 if gelu else 1.25) * np.abs(arg)
                slope = p + v * p * q * D
                # p's own error; that of 1 - p (p's, and a rounding), of a and of the products
                es = p * (e * q + 6) + np.abs(v * p * D) * (q * (2 * e + 12) + p * (q * e + 6))
            else:
                slope = np.where(v < 0, 0.0, 2 * v) if act == nv.NVFP4_ACT_RELU2 else np.ones_like(v)
                es = 0.0 * v
            ref = f64(dy) * u * slope
            close(f64(dg), ref, np.abs(ref) * (hs + 3 * U) + np.abs(f64(dy) * u) * (es * U * (1 + hs))
                  + floor * np.abs(f64(dy)), f"dgate of {act}")


@pytest.mark.parametrize("dt", [BF, F32])
def test_every_exponent_is_kept(dt):
    """Blocks of every magnitude of the type, from subnormal ones on: the smallest byte that
    holds them, saturation at 127 above its range, and restored values."""
    torch = gpuio.torch_cuda()
    rng = np.random.default_rng(3)
    e = np.arange(-149, 128)
    a = rng.uniform(-1, 1, (len(e), 64))
    a[:, 0] = 1.0       # exactly a power of two
    a[:, 32] = 127 / 64  # the largest that the byte below holds
    a[:, 33:] *= 1.98
    x64 = a * 2.0 ** e[:, None]
    x = torch.from_numpy(np.clip(x64, -3.4e38, 3.4e38)).float().cuda()
    x = x if dt == F32 else torch.where(torch.isinf(x.bfloat16()), torch.full_like(x, 3.38e38), x).bfloat16()
    rows, cols = x.shape
    g, codes, scales = kept_buffers(rows, cols)
    out = torch.empty((rows, cols), device="cuda")
    nv.nvfp4_gated_act(nv.NVFP4_ACT_NONE, x, None, dt, rows, cols, cols, 0, None, 0, codes, scales, None, None)
    nv.nvfp4_gated_act_backward(nv.NVFP4_ACT_NONE, codes, scales, None, None, None, F32, rows, cols, 0, None, 0, None, 0,
                                out, cols)
    torch.cuda.synchronize()
    g.check()
    q, s = kept64(f64(x))
    c, b = codes.cpu().numpy(), scales.cpu().numpy()
    assert np.array_equal(b, s) and np.array_equal(c, q)
    assert np.array_equal(f64(out), held64(c, b))


def test_blocks_that_hold_infinities_or_nan():
    torch = gpuio.torch_cuda()
    x = torch.ones((2, 96), device="cuda", dtype=torch.bfloat16)
    x[0, 40], x[1, 95] = float("inf"), float("nan")
    g, codes, scales = kept_buffers(2, 96)
    y, dg = torch.empty_like(x), torch.empty_like(x)
    nv.nvfp4_gated_act(nv.NVFP4_ACT_SILU, x, None, BF, 2, 96, 96, 0, y, 96, codes, scales, None, None)
    nv.nvfp4_gated_act_backward(nv.NVFP4_ACT_SILU, codes, scales, None, None, torch.ones_like(x), BF, 2, 96, 96, dg, 96,
                                None, 0, None, 0)
    # 1.0 is 64 * 2^(127 - 133); under byte 126 its code would be 128
    assert scales.cpu().tolist() == [[127, 255, 127], [127, 127, 255]]
    c = codes.cpu().numpy()
    assert (c[0, 32:64] == 0).all() and (c[1, 64:] == 0).all() and (c[0, :32] == 64).all()
    nan = torch.isnan(dg).cpu().numpy()
    assert nan[0, 32:64].all() and nan[1, 64:].all() and nan.sum() == 64
    assert float(y[0, 40]) == float("inf") and bool(torch.isnan(y[1, 95])) and int(torch.isnan(y).sum()) == 1


def test_in_place():
    """Outputs may be inputs of their own size, also where rows are read more than once."""
    torch = gpuio.torch_cuda()
    for dt, rows, cols in ((BF, 5, 300), (BF, 3, 70001), (F32, 3, 20481)):
        t = torch.bfloat16 if dt == BF else torch.float32
        gen = torch.Generator(device="cuda").manual_seed(cols)
        rnd = lambda *s: torch.randn(*s, generator=gen, device="cuda").to(t)  # noqa: E731
        x, r, gate, dy, dh, one = rnd(rows, cols), rnd(rows, cols), rnd(rows, cols), rnd(rows, cols), rnd(rows, cols), rnd(cols)
        stats = [torch.empty(rows, device="cuda") for _ in range(2)]

        def norms(h, y, res, xx):
            nv.nvfp4_block_norms(xx, res, gate, dt, rows, cols, cols, cols, cols, 1, one, one, dt, EPS, 0.5, h, cols, y,
                                 cols, None, 0, None, *stats)
            return h.clone(), y.clone()
        want = norms(torch.empty_like(x), torch.empty_like(x), r, x)
        h, xx = r.clone(), x.clone()
        got = norms(h, xx, h, xx)
        assert all(torch.equal(a, b) for a, b in zip(want, got))
        size = nv.nvfp4_block_norms_backward_workspace_size(rows, cols)
        ws = torch.empty(size, dtype=torch.uint8, device="cuda")

        def back(dy, dh, gate, dx, dr, dg):
            sums = [torch.empty(cols, device="cuda") for _ in range(2)]
            nv.nvfp4_block_norms_backward(dy, dh, h, x, gate, dt, rows, cols, *([cols] * 5), 1, one, one, dt, *stats, 0.5,
                                          dx, cols, dr, cols, dg, cols, *sums, ws)
            return [v.clone() for v in (dx, dr, dg, *sums)]
        want = back(dy, dh, gate, *(torch.empty_like(x) for _ in range(3)))
        a, b, c = dy.clone(), dh.clone(), gate.clone()
        got = back(a, b, c, a, b, c)
        assert all(torch.equal(u, v) for u, v in zip(want, got))
