"""The product of 8-bit integers and the quantization of its input against plain
computations on the host.

The product's sum is exact, and its two scalings are FP32 products in a fixed
order, so that FP32 results are compared bit for bit, BF16 results with that FP32
value rounded to nearest even.  Codes of a tensor are compared bit for bit with
their definition's FP32 operations; those of an activation or a norm, whose values
may be off by a few roundings, may lie one code beside the definition's where the
64-bit value is that near a border."""
import numpy as np
import pytest

import bit_microscaled_quantized_amd as nv
from tests import gpuio
from tests.test_gpu_norm import F32, BF, Tensors, data, f64

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
f32 = np.float32


def up16(n):
    return (n + 15) // 16 * 16


def codes_of(v):
    """Codes and scales of FP32 rows by their definition, each operation in FP32."""
    top = np.abs(v).max(1).astype(f32)
    ok = np.isfinite(top)
    live = ok & (top >= f32(2.0 ** -100))
    with np.errstate(all="ignore"):
        inv = np.where(live, f32(127) / np.where(live, top, f32(1)), f32(0)).astype(f32)
        scale = np.where(live, top / f32(127), f32(0)).astype(f32)
        q = np.rint((v * inv[:, None]).astype(f32))
    q[~ok] = 0
    scale[~ok] = np.nan
    return q.astype(np.int8), scale


def code_buffers(rows, cols, pad=0):
    torch = gpuio.torch_cuda()
    g = gpuio.Guarded()
    ld = up16(cols) + pad
    return g, g.alloc((max(rows, 1), ld), torch.int8, fill=55), g.alloc((max(rows, 1),), torch.float32, fill=5.0)


def check_pads(g, codes, rows, cols):
    g.check()
    c = codes.cpu().numpy()
    assert (c[:rows, cols:up16(cols)] == 0).all(), "codes past the columns are not zero"
    assert (c[:rows, up16(cols):] == 55).all(), "codes past the padding were written"
    return c[:rows, :cols]


SHAPES = [(0, 8), (1, 1), (1, 2), (5, 15), (3, 16), (2, 31), (33, 32), (17, 33), (40, 127), (7, 128), (65, 129),
          (5, 255), (16, 513), (1030, 1025), (3, 2049), (130, 5120), (9, 5119), (2, 20479), (2, 40960), (2, 40961),
          (1, 70001)]


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("dt,pad,off", [(BF, 0, 0), (BF, 3, 1), (F32, 0, 0), (F32, 5, 3)])
def test_quantize(rows, cols, dt, pad, off):
    torch = gpuio.torch_cuda()
    rng = np.random.default_rng(rows * 31 + cols)
    a = data(rng, rows, cols)
    if rows > 2:
        a[1] = 0.0
        a[2] *= 2.0 ** -103  # below and around the smallest row that has codes
        a[0] *= 2.0 ** 100
    T = Tensors(rows, cols, dt, pad, off)
    x = T.put(a)
    g, codes, scales = code_buffers(rows, cols, 16 * (pad > 0))
    nv.nvfp4_int8_quantize(x, dt, rows, cols, T.ld, codes, codes.stride(0), scales)
    torch.cuda.synchronize()
    q, s = codes_of(x.float().cpu().numpy()) if rows else (np.zeros((0, cols), np.int8), np.zeros(0, f32))
    assert np.array_equal(check_pads(g, codes, rows, cols), q)
    assert np.array_equal(scales.cpu().numpy()[:rows], s)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("cols", [40, 5120, 50000])
def test_quantize_infinities_and_nan(dt, cols):
    torch = gpuio.torch_cuda()
    x = torch.ones((5, cols), device="cuda", dtype=torch.bfloat16 if dt == BF else torch.float32)
    x[1, 7], x[2, cols - 1], x[3, 0] = float("inf"), float("nan"), -float("inf")
    g, codes, scales = code_buffers(5, cols)
    nv.nvfp4_int8_quantize(x, dt, 5, cols, cols, codes, codes.stride(0), scales)
    torch.cuda.synchronize()
    c, s = check_pads(g, codes, 5, cols), scales.cpu().numpy()
    assert (c[[0, 4]] == 127).all() and (c[1:4] == 0).all()
    assert np.isnan(s[1:4]).all() and (s[[0, 4]] == f32(1) / f32(127)).all()


def act64(act, v):
    """(act(v), relative error of its FP32 form in units of u away from zero).  The logistic
    function's: 1.25 |arg| for the exponent's product, 5 for the two instructions' 1 ulp each
    and two roundings, each weighted by at most 1; GELU's argument has 3 roundings more."""
    if act == nv.NVFP4_ACT_SILU:
        arg = v
        extra = 1.25
    elif act == nv.NVFP4_ACT_GELU:
        arg = np.sqrt(8 / np.pi) * (v + 0.044715 * v ** 3)
        extra = 4.25
    elif act == nv.NVFP4_ACT_RELU2:
        return np.where(v < 0, 0.0, v) ** 2, np.full(v.shape, 2.0)
    else:
        return v, np.zeros(v.shape)
    with np.errstate(over="ignore"):
        p = 1 / (1 + np.exp(-arg))
    return v * p, 7.0 + extra * np.abs(arg)


@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 33), (65, 129), (1030, 1025), (48, 20480), (2, 50001)])
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("act", range(4))
@pytest.mark.parametrize("gated", [False, True])
def test_quantize_gated(rows, cols, dt, act, gated):
    torch = gpuio.torch_cuda()
    rng = np.random.default_rng(rows * 31 + cols + act)
    T = Tensors(rows, cols, dt, 3, 1)
    gate, up = T.put(data(rng, rows, cols)), T.put(data(rng, rows, cols))
    g, codes, scales = code_buffers(rows, cols)
    nv.nvfp4_int8_quantize_gated(act, gate, up if gated else None, dt, rows, cols, T.ld, T.ld, codes, codes.stride(0),
                                 scales)
    torch.cuda.synchronize()
    v, rel = act64(act, f64(gate))
    if gated:
        v, rel = v * f64(up), rel + 1
    tol = np.abs(v) * rel * U + 1e-36
    top, worst = np.abs(v).max(1), (np.abs(v) + tol).max(1)
    step = np.maximum(top / 127, 1e-300)
    s = scales.cpu().numpy().astype(np.float64)
    assert (np.abs(s - top / 127) <= (worst - top) / 127 + 2 * U * top / 127).all()
    # of the code before rounding: the value's error, the largest magnitude's, two roundings
    off = tol / step[:, None] + 127 * ((worst - top) / np.maximum(top, 1e-300))[:, None] + 127 * 3 * U
    c = check_pads(g, codes, rows, cols).astype(np.float64)
    assert (np.abs(c - v / step[:, None]) <= 0.5 + off).all()


def product(a, sa, b, sb):
    z = (a.astype(np.float64) @ b.astype(np.float64).T).astype(f32)  # exact below 2^53, then one rounding
    return ((z * sb[None, :]).astype(f32) * sa[:, None]).astype(f32)


SIZES = [(0, 8, 16), (1, 1, 16), (1, 5, 32), (1, 16, 48), (2, 17, 64), (3, 64, 112), (1, 300, 2048), (5, 129, 1040),
         (15, 257, 512), (16, 512, 4096), (17, 100, 5120), (31, 1000, 336), (33, 640, 1536), (48, 320, 20480),
         (63, 65, 8192), (64, 64, 256), (65, 255, 768), (100, 1003, 2064), (128, 128, 1024), (129, 130, 272),
         (200, 2050, 144), (256, 256, 512), (257, 4999, 2048), (300, 513, 640), (511, 127, 131056), (1000, 700, 1280),
         (2, 3, 131056), (2049, 2305, 80)]


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("layout", ["packed", "padded", "no workspace"])
def test_product(M, N, K, dt, layout):
    torch = gpuio.torch_cuda()
    rng = np.random.default_rng(M * 7 + N * 3 + K)
    pa, pb, pc = (0, 0, 0) if layout == "packed" else (16, 48, 5)
    a, b = (rng.integers(-128, 128, (max(n, 1), K + p), dtype=np.int8) for n, p in ((M, pa), (N, pb)))
    sa, sb = (rng.uniform(1e-3, 2e-3, max(n, 1)).astype(f32) for n in (M, N))
    g = gpuio.Guarded()
    t = torch.bfloat16 if dt == BF else torch.float32
    c = g.alloc((max(M, 1), N + pc), t, fill=7.0)
    ws_bytes = nv.nvfp4_int8_gemm_workspace_size(M, N, K)
    ws = None if layout == "no workspace" else g.alloc((ws_bytes + 16,), torch.uint8)
    ta, tb, tsa, tsb = (gpuio.to_dev(v) for v in (a, b, sa, sb))
    for _ in range(2):  # a workspace's old contents do not matter
        nv.nvfp4_int8_gemm(M, N, K, ta, K + pa, tsa, tb, K + pb, tsb, c, dt, N + pc, ws, 0 if ws is None else ws_bytes)
    torch.cuda.synchronize()
    g.check()
    ref = torch.from_numpy(product(a[:M, :K], sa[:M], b[:N, :K], sb[:N])).to(t)
    got = c.cpu()
    assert bool((got[:, N:] == 7.0).all()), "a gap between rows was written"
    bad = got[:M, :N] != ref
    assert not bool(bad.any()), f"{int(bad.sum())} of {M * N} differ, first at {bad.nonzero()[0].tolist()}"


def test_product_of_the_largest_sums():
    torch = gpuio.torch_cuda()
    K = 131056
    one = torch.ones(3, device="cuda")
    for va, vb in ((-128, -128), (127, -128), (127, 127)):
        a = torch.full((3, K), va, dtype=torch.int8, device="cuda")
        b = torch.full((2, K), vb, dtype=torch.int8, device="cuda")
        c = torch.empty((3, 2), device="cuda")
        nv.nvfp4_int8_gemm(3, 2, K, a, K, one, b, K, one, c, F32, 2)
        assert (c.cpu().numpy() == f32(va * vb * K)).all()


def test_product_carries_scales_that_are_not_numbers():
    torch = gpuio.torch_cuda()
    for M in (3, 70, 300):
        a = torch.zeros((M, 64), dtype=torch.int8, device="cuda")
        b = torch.ones((40, 64), dtype=torch.int8, device="cuda")
        sa, sb = torch.ones(M, device="cuda"), torch.ones(40, device="cuda")
        sa[1] = float("nan")
        sb[5] = float("inf")
        c = torch.empty((M, 40), device="cuda")
        nv.nvfp4_int8_gemm(M, 40, 64, a, 64, sa, b, 64, sb, c, F32, 40)
        nan = torch.isnan(c).cpu().numpy()
        want = np.zeros((M, 40), bool)
        want[1], want[:, 5] = True, True
        assert np.array_equal(nan, want) and (c.cpu().numpy()[~want] == 0).all()


def test_quantized_tensor_times_weight():
    """The two calls together: within the roundings to 8 bits of the product in 64 bits."""
    torch = gpuio.torch_cuda()
    rng = np.random.default_rng(5)
    M, N, K = 37, 300, 1000
    x, w = rng.normal(size=(M, K)), rng.normal(size=(N, K)) * 0.02
    ops = []
    for v in (x, w):
        t = torch.from_numpy(v).float().cuda()
        codes = torch.empty((v.shape[0], up16(K)), dtype=torch.int8, device="cuda")
        scales = torch.empty(v.shape[0], device="cuda")
        nv.nvfp4_int8_quantize(t, F32, v.shape[0], K, K, codes, up16(K), scales)
        ops.append((codes, scales))
    (a, sa), (b, sb) = ops
    c = torch.empty((M, N), device="cuda")
    nv.nvfp4_int8_gemm(M, N, up16(K), a, up16(K), sa, b, up16(K), sb, c, F32, N)
    # each factor is off by at most half a step of its row (and its code's FP32 roundings)
    half = (0.5 + 400 * U)
    ex, ew = (np.abs(v).max(1) / 127 * half for v in (x, w))
    tol = (np.abs(x).sum(1)[:, None] * ew[None, :] + ex[:, None] * np.abs(w).sum(1)[None, :]
           + K * ex[:, None] * ew[None, :])
    assert (np.abs(f64(c) - x @ w.T) <= tol + 1e-6).all()
