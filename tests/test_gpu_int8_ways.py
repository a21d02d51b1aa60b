"""One size and more for each way that the product of 8-bit integers takes: few tokens with
their codes read by each wave or shared, whole K or in parts; every tile size with an
even number of whole stages, with any, with less than one; tiles behind the last full
round in parts.  Results are compared bit for bit: the sums are exact in 64 bits, then
three FP32 roundings in the definition's order."""
import pytest

import bit_microscaled_quantized_amd as nv
from tests import gpuio

pytestmark = pytest.mark.gpu

F32, BF = nv.NVFP4_F32, nv.NVFP4_BF16


def product(torch, a, sa, b, sb):
    z = (a.double() @ b.double().t().contiguous()).float()
    return (z * sb[None, :]) * sa[:, None]


@pytest.mark.parametrize("M,N,K,split", [
    # few tokens: each wave for itself, in four and in eight slices of K, whole and in parts
    (1, 12000, 512, False), (3, 10240, 5120, False), (8, 20000, 272, False), (1, 100, 20480, True), (7, 1000, 40976, True),
    (16, 1024, 5120, False), (12, 333, 20464, True), (2, 40, 131056, True), (1, 65, 304, False), (5, 16385, 1040, False),
    # shared by four waves, whole and in parts, every number of tiles of tokens
    (16, 10000, 4096, True), (11, 41000, 1040, False), (17, 300, 512, False), (32, 5120, 2064, False), (33, 70, 9008, True),
    (48, 41100, 1024, False), (49, 1000, 784, False), (64, 5120, 20480, True), (64, 64, 131056, True), (50, 130, 16, False),
    # 64 x 64 tiles: less than a stage, whole stages, any, in parts
    (65, 100, 16, False), (300, 257, 112, False), (100, 2048, 512, False), (257, 4999, 2048, False), (130, 1000, 400, False),
    (128, 1024, 5120, True), (70, 300, 20000, True), (66, 65, 128, False), (100, 100, 256, False), (90, 200, 144, False),
    # 128 x 128
    (256, 20480, 512, False), (1024, 5120, 1040, False), (128, 5120, 20480, True), (250, 5000, 20464, True),
    (8000, 700, 1280, False), (513, 6000, 3088, False),
    # 256 x 256
    (2048, 5120, 2560, False), (2000, 5000, 5136, False), (4096, 5120, 4096, False), (4095, 5117, 4112, False),
    (1024, 5120, 20480, True), (1000, 5111, 20464, True), (4097, 4097, 1296, False),
])
@pytest.mark.parametrize("dt", [BF, F32])
def test_every_way(M, N, K, split, dt):
    torch = gpuio.torch_cuda()
    g = torch.Generator(device="cuda").manual_seed(M + N + K)
    rnd = lambda r: torch.randint(-127, 128, (r, K), generator=g, device="cuda", dtype=torch.int32).to(torch.int8)  # noqa: E731
    a, b = rnd(M), rnd(N)
    sa, sb = (0.001 + torch.rand(n, generator=g, device="cuda") for n in (M, N))
    size = nv.nvfp4_int8_gemm_workspace_size(M, N, K)
    assert (size > 0) == split
    guard = gpuio.Guarded()
    t = torch.bfloat16 if dt == BF else torch.float32
    c = guard.alloc((M, N), t, fill=7.0)
    ws = guard.alloc((max(size, 16),), torch.uint8)
    nv.nvfp4_int8_gemm(M, N, K, a, K, sa, b, K, sb, c, dt, N, ws, size)
    torch.cuda.synchronize()
    guard.check()
    want = product(torch, a, sa, b, sb).to(t)
    assert torch.equal(c, want)
    if split:  # without the parts
        c.fill_(7.0)
        nv.nvfp4_int8_gemm(M, N, K, a, K, sa, b, K, sb, c, dt, N, ws, size - 16)
        assert torch.equal(c, want)


def test_rows_far_apart():
    """Operands whose rows lie up to 2^23 bytes apart: offsets beyond 2^32 within a tile's rows' range."""
    torch = gpuio.torch_cuda()
    ld = (1 << 23) - 16
    for M, N in ((3, 600), (600, 70), (40, 300)):
        g = torch.Generator(device="cuda").manual_seed(M)
        big = torch.zeros(max(M, N) * ld, dtype=torch.int8, device="cuda").view(max(M, N), ld)
        big[:, :272] = torch.randint(-127, 128, (max(M, N), 272), generator=g, device="cuda").to(torch.int8)
        a, b = big[:M, :272], big[:N, :272]
        one = torch.ones(max(M, N), device="cuda")
        c = torch.empty((M, N), device="cuda")
        nv.nvfp4_int8_gemm(M, N, 272, a, ld, one, b, ld, one, c, F32, N)
        assert torch.equal(c, product(torch, a, one[:M], b, one[:N]))
        del big


def test_a_wide_output():
    """Rows of an output 2^25 elements apart: places beyond 2^31 elements."""
    torch = gpuio.torch_cuda()
    a = torch.ones((70, 16), dtype=torch.int8, device="cuda")
    b = torch.ones((1 << 20, 16), dtype=torch.int8, device="cuda")
    sa = torch.arange(70, device="cuda").float()
    sb = torch.ones(1 << 20, device="cuda")
    c = torch.empty((70, 1 << 25), dtype=torch.bfloat16, device="cuda")
    nv.nvfp4_int8_gemm(70, 1 << 20, 16, a, 16, sa, b, 16, sb, c, BF, 1 << 25)
    want = (16.0 * sa).bfloat16()
    assert bool((c[:, :1 << 20] == want[:, None]).all())
