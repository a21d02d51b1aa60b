"""The 8-bit block operators where offsets pass 32 bits: rows at the end of tensors of almost
2^32 elements have the results of a call on those rows alone."""
import pytest
import torch

import bit_microscaled_quantized_amd as nv
from bit_microscaled_quantized_amd import blocks

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
TAIL = 1030  # rows enough for the lanes a row of the large call


def rand(rows, cols, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.empty(rows, cols, device="cuda", dtype=BF)
    x[:-TAIL] = torch.randn(1, cols, generator=g, device="cuda").to(BF)
    x[-TAIL:] = torch.randn(TAIL, cols, generator=g, device="cuda").to(BF)
    return x


@pytest.fixture(autouse=True)
def room():
    free, _ = torch.cuda.mem_get_info()
    if free < 120 << 30:
        pytest.skip("needs 120 GB of device memory")
    yield
    torch.cuda.empty_cache()


@pytest.mark.parametrize("rows,cols", [(838000, 5120), (42000, 102001)])
def test_norms(rows, cols):
    assert 2 ** 31 < rows * cols < 2 ** 32
    x, r = rand(rows, cols, 1), rand(rows, cols, 2)
    gains = [torch.rand(cols, device="cuda").add_(0.5).to(BF) for _ in range(2)]
    with torch.no_grad():
        h, y = blocks.block_norms(x, r, *gains, scale=0.5)
        h2, y2 = blocks.block_norms(x[-TAIL:], r[-TAIL:], *gains, scale=0.5)
        assert torch.equal(h[-TAIL:], h2) and torch.equal(y[-TAIL:], y2)
        assert torch.equal(y[0], y[-TAIL - 1])
        del y
        _, codes, scales = blocks.block_norms_int8(x, r, *gains, scale=0.5)
        _, codes2, scales2 = blocks.block_norms_int8(x[-TAIL:], r[-TAIL:], *gains, scale=0.5)
        assert torch.equal(codes[-TAIL:], codes2) and torch.equal(scales[-TAIL:], scales2)
        assert torch.equal(codes[0], codes[-TAIL - 1])


@pytest.mark.parametrize("rows,cols", [(838000, 5120), (42000, 102001)])
def test_norms_backward(rows, cols):
    x, dy = rand(rows, cols, 3), rand(rows, cols, 4)
    gains = [torch.rand(cols, device="cuda").add_(0.5).to(BF) for _ in range(2)]

    def grads(x, dy):
        x = x.detach().requires_grad_()
        h, y = blocks.block_norms(x, None, *gains, scale=0.5)
        return torch.autograd.grad(y, x, dy)[0]
    assert torch.equal(grads(x, dy)[-TAIL:], grads(x[-TAIL:], dy[-TAIL:]))


@pytest.mark.parametrize("rows,cols", [(209000, 20480), (4200000, 1021)])
def test_activation(rows, cols):
    gate, up = rand(rows, cols, 5), rand(rows, cols, 6)
    with torch.no_grad():
        assert torch.equal(blocks.gated_act(gate, up)[-TAIL:], blocks.gated_act(gate[-TAIL:], up[-TAIL:]))
        codes, scales = blocks.int8_quantize_gated(gate, up)
        codes2, scales2 = blocks.int8_quantize_gated(gate[-TAIL:], up[-TAIL:])
        assert torch.equal(codes[-TAIL:], codes2) and torch.equal(scales[-TAIL:], scales2)
    del up, codes
    kept = blocks.keep8(gate)
    kept2 = blocks.keep8(gate[-TAIL:])
    assert all(torch.equal(a[-TAIL:], b) for a, b in zip(kept, kept2))
    assert torch.equal(blocks.restore8(*kept)[-TAIL:], blocks.restore8(*kept2))


@pytest.mark.parametrize("M,N,K", [(2 ** 23, 4096, 16), (1030000, 16640, 256), (64, 2 ** 24 - 1, 272), (2 ** 24 - 1, 33, 400)])
def test_product(M, N, K):
    """M N up to 2^35: the output's last rows and columns."""
    g = torch.Generator(device="cuda").manual_seed(M)
    a, b = (torch.empty(r, K, device="cuda", dtype=torch.int8).random_(-127, 128, generator=g) for r in (M, N))
    sa, sb = (0.001 + torch.rand(r, generator=g, device="cuda") for r in (M, N))
    c = blocks.int8_matmul(a, sa, b, sb)
    for rows in (slice(0, 70), slice(M // 2, M // 2 + 70), slice(max(M - 70, 0), M)):
        for cols in (slice(0, 70), slice(N // 2, N // 2 + 70), slice(max(N - 70, 0), N)):
            want = (a[rows].double() @ b[cols].double().t().contiguous()).float() * sb[cols] * sa[rows, None]
            assert torch.equal(c[rows, cols], want.to(BF))


def test_product_of_wide_strides():
    """Leading dimensions of almost 2^23: a tile's rows lie almost 2^31 bytes apart."""
    ld = 2 ** 23 - 16
    for M, N, K in ((300, 257, 400), (33, 70, 400)):
        g = torch.Generator(device="cuda").manual_seed(M)
        wide = [torch.zeros(r, ld, device="cuda", dtype=torch.int8) for r in (M, N)]
        a, b = (w[:, 160:160 + K] for w in wide)
        for t in (a, b):
            t.copy_(torch.empty(t.shape, device="cuda", dtype=torch.int8).random_(-127, 128, generator=g))
        sa, sb = torch.rand(M, device="cuda"), torch.rand(N, device="cuda")
        c = torch.empty(M, N, device="cuda")
        nv.nvfp4_int8_gemm(M, N, K, a, ld, sa, b, ld, sb, c, nv.NVFP4_F32, N, None, 0)
        want = (a.double() @ b.double().t().contiguous()).float() * sb * sa[:, None]
        assert torch.equal(c, want)
        assert torch.equal(blocks.int8_matmul(a, sa, b, sb, torch.float32), want)
