"""Edges of the 8-bit block operators: the largest activations, layers whose model changes
its type, workspaces that two captured graphs share, the LDS that a large tile takes."""
import pytest
import torch

import bit_microscaled_quantized_amd as nv
from bit_microscaled_quantized_amd import blocks

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,N,K", [
    # tiles of 256 and of 128 behind full rounds, or all of them, in parts; K a multiple of two stages, and not
    (4096, 5120, 20480), (4095, 5117, 20464), (512, 5120, 20480), (500, 5111, 20464), (100, 5111, 20464),
])
def test_products_in_parts(M, N, K):
    g = torch.Generator(device="cuda").manual_seed(M + K)
    a, b = (torch.randint(-127, 128, (r, K), generator=g, device="cuda", dtype=torch.int32).to(torch.int8) for r in (M, N))
    sa, sb = (0.001 + torch.rand(r, generator=g, device="cuda") for r in (M, N))
    assert nv.nvfp4_int8_gemm_workspace_size(M, N, K) > 0
    want = ((a.double() @ b.double().t().contiguous()).float() * sb * sa[:, None]).to(torch.bfloat16)
    assert torch.equal(blocks.int8_matmul(a, sa, b, sb), want)
    c = torch.empty_like(want)
    nv.nvfp4_int8_gemm(M, N, K, a, K, sa, b, K, sb, c, nv.NVFP4_BF16, N, None, 0)  # without a workspace
    assert torch.equal(c, want)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("act", ["none", "silu", "gelu", "relu2"])
def test_slopes_of_the_largest_activations(dtype, act):
    """Where v^2 (or exp(-v)) overflows: the slopes are 1 and 0 exactly, relu2's 2 v."""
    v = torch.tensor([1e18, 1e19, 1.8e19, 2e19, 1e25, 1e30, 1e37, 1e38, 3e38], dtype=dtype, device="cuda")
    v = torch.cat([v, -v]).view(-1, 1).repeat(1, 32).requires_grad_()  # a block each
    y = blocks.gated_act(v, None, act)
    y.backward(torch.ones_like(y))
    at = blocks.restore8(*blocks.keep8(v.detach()), dtype=torch.float32)
    up = at > 0
    slope = {"none": torch.ones_like(at), "silu": up.float(), "gelu": up.float(), "relu2": 2 * at.clamp(min=0)}[act]
    assert torch.equal(v.grad, slope.to(dtype))


def test_a_layer_keeps_its_scales_in_fp32():
    torch.manual_seed(0)
    layer = blocks.Int8Linear(torch.randn(40, 48, device="cuda"))
    x = torch.randn(5, 48, device="cuda", dtype=torch.bfloat16)
    want = layer(x)
    moved = torch.nn.Sequential(layer).to(torch.bfloat16)
    assert layer.scales.dtype == torch.float32 and layer.codes.dtype == torch.int8
    assert torch.equal(moved(x), want)
    assert torch.equal(layer.half()(x), want)


def test_scales_that_need_a_gradient_are_refused():
    codes, scales = blocks.int8_quantize(torch.ones(4, 32, device="cuda"))
    with pytest.raises(RuntimeError, match="no gradient"):
        blocks.int8_matmul(codes, scales.requires_grad_(), codes, scales.detach())


@pytest.mark.parametrize("M,N,K", [
    (17, 33000, 1040), (33, 4100, 8208), (49, 70000, 496), (32, 2300, 20464), (60, 1700, 20464), (64, 512, 131056),
    (33, 3000, 11200), (17, 2 ** 21, 16), (50, 8191, 4112), (16, 8000, 4112)])
def test_large_weights_stream_past_shared_tokens(M, N, K):
    """Weights of 2^25 codes and more, whole and in parts, K that ends inside a stage, N inside a group of rows."""
    g = torch.Generator(device="cuda").manual_seed(N)
    a, b = (torch.empty(r, K, device="cuda", dtype=torch.int8).random_(-127, 128, generator=g) for r in (M, N))
    sa, sb = (0.001 + torch.rand(r, generator=g, device="cuda") for r in (M, N))
    want = (a.double() @ b.double().t().contiguous()).float() * sb * sa[:, None]
    assert torch.equal(blocks.int8_matmul(a, sa, b, sb, torch.float32), want)
    c = torch.empty(M, N, device="cuda", dtype=torch.bfloat16)
    nv.nvfp4_int8_gemm(M, N, K, a, K, sa, b, K, sb, c, nv.NVFP4_BF16, N, None, 0)  # without a workspace
    assert torch.equal(c, want.to(torch.bfloat16))


def test_two_graphs_share_a_workspace():
    """Calls in two captured graphs with one workspace, replayed in turn on one stream, with
    eager work between: the same results as alone."""
    torch.manual_seed(1)
    gemms = []
    for M, N, K in ((48, 512, 4096), (130, 512, 8192), (1, 512, 16384)):
        a = torch.randint(-127, 128, (M, K), dtype=torch.int8, device="cuda")
        b = torch.randint(-127, 128, (N, K), dtype=torch.int8, device="cuda")
        sa, sb = torch.rand(M, device="cuda"), torch.rand(N, device="cuda")
        gemms.append((M, N, K, a, sa, b, sb, torch.empty(M, N, device="cuda")))
    size = max(nv.nvfp4_int8_gemm_workspace_size(*g[:3]) for g in gemms)
    assert min(nv.nvfp4_int8_gemm_workspace_size(*g[:3]) for g in gemms) > 0
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")

    def run(g):
        M, N, K, a, sa, b, sb, c = g
        nv.nvfp4_int8_gemm(M, N, K, a, K, sa, b, K, sb, c, nv.NVFP4_F32, N, ws)
    want = []
    for g in gemms:
        run(g)
        want.append(g[-1].clone())
        exact = (g[3].double() @ g[5].double().t()).float() * g[6] * g[4][:, None]
        assert torch.equal(want[-1], exact)
    torch.cuda.synchronize()
    graphs = []
    for some in (gemms[:2], gemms[1:]):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            for g in some:
                run(g)
        graphs.append((graph, some))
    for n in range(4):
        for g in gemms:
            g[-1].fill_(-1.0)
        for graph, _ in graphs if n % 2 else graphs[::-1]:
            graph.replay()
            ws.random_(0, 256)
        torch.cuda.synchronize()
        for g, w in zip(gemms, want):
            assert torch.equal(g[-1], w)


def test_a_backward_pass_in_a_graph():
    """Forward and backward of a block's norms and activation captured together, replayed
    with new inputs in the same buffers."""
    torch.manual_seed(2)
    rows, cols = 70, 264

    def fresh():
        return torch.randn(rows, cols, device="cuda", dtype=torch.bfloat16)
    x, r, up = (fresh().requires_grad_() for _ in range(3))
    gains = [torch.rand(cols, device="cuda").add_(0.5).to(torch.bfloat16).requires_grad_() for _ in range(3)]
    leaves = [x, r, up, *gains]

    def grads():
        h, y = blocks.block_norms(x, r, gains[0], gains[1], gains[2], 0.5)
        z = blocks.gated_act(y, up, "gelu")
        return torch.autograd.grad((z, h), leaves, (torch.ones_like(z), torch.ones_like(h)))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        grads()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = grads()
    for _ in range(3):
        with torch.no_grad():
            for t in (x, r, up):
                t.copy_(fresh())
        graph.replay()
        torch.cuda.synchronize()
        for got, want in zip(out, grads()):
            assert torch.equal(got, want)


@pytest.mark.parametrize("rows", [0, 1, 7])
def test_rows_of_codes_start_on_lines(rows):
    """The codes' buffer is wider than the codes; a module's moves, copies and states keep its results."""
    torch.manual_seed(3)
    x = torch.randn(rows, 88, device="cuda", dtype=torch.bfloat16)
    codes, scales = blocks.int8_quantize(x)
    assert codes.shape == (rows, 96) and codes.stride() == (128, 1) and codes.data_ptr() % 128 == 0
    assert not codes[:, 88:].any()
    layer = blocks.Int8Linear(torch.randn(40, 88, device="cuda"))
    want = layer(x)
    exact = (codes.double() @ layer.codes.double().t().contiguous()).float() * layer.scales * scales[:, None]
    assert torch.equal(want, exact.to(torch.bfloat16))
    there = layer.cpu().cuda()
    assert there.codes.stride(0) == 128 and torch.equal(there(x), want)
    other = blocks.Int8Linear(torch.randn(40, 88, device="cuda"))
    other.load_state_dict(layer.state_dict())
    assert other.codes.stride(0) == 128 and torch.equal(other(x), want)
    assert torch.equal(blocks.int8_matmul(codes.contiguous(), scales, layer.codes.contiguous(), layer.scales, torch.bfloat16), want)
