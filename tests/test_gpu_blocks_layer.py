"""The layer over the operators of a residual block in eight bits: gradients against
64-bit autograd and against differences, the operators' use together in training and
serving, under graph capture and on two streams, and what it refuses."""
import pytest

from tests import gpuio

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def rms(torch, v, gamma, eps=1e-5):
    return v * torch.rsqrt(v.square().mean(-1, keepdim=True) + eps) * gamma


def plain_norms(torch, x, residual, post, pre, gate, scale, sigmoid):
    o = rms(torch, x, post)
    if gate is not None:
        o = o * (torch.sigmoid(gate) if sigmoid else gate)
    h = scale * o + (0 if residual is None else residual)
    return h, rms(torch, h, pre)


def plain_act(torch, act, v):
    if act == "silu":
        return v * torch.sigmoid(v)
    if act == "gelu":
        return torch.nn.functional.gelu(v, approximate="tanh")
    return torch.relu(v).square() if act == "relu2" else v


def rnd(torch, seed, *shape, dtype=None, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = torch.randn(*shape, generator=g, device="cuda") * scale
    return t if dtype is None else t.to(dtype)


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("kind", [None, "channel", "token"])
@pytest.mark.parametrize("residual", [False, True])
def test_norms_gradients(dtype, kind, residual):
    """Against FP64 autograd of the formulas at the same (rounded) leaves.  h and dy are rounded to the tensors'
    type between the passes, gradients once more: four such roundings and the FP32 sums' 2^-14 added as norms."""
    torch = gpuio.torch_cuda()
    from bit_microscaled_quantized_amd.blocks import block_norms
    t = getattr(torch, dtype)
    B, S, H = 3, 21, 520
    leaves = [rnd(torch, 1, B, S, H, dtype=t), rnd(torch, 2, B, S, H, dtype=t) if residual else None,
              (1 + rnd(torch, 3, H, scale=0.2)).to(t), (1 + rnd(torch, 4, H, scale=0.2)).to(t),
              None if kind is None else rnd(torch, 5, *((H,) if kind == "channel" else (B, S, H)), dtype=t)]
    wy, wh = rnd(torch, 6, B, S, H, dtype=t), rnd(torch, 7, B, S, H, dtype=t)
    mine = [None if v is None else v.clone().requires_grad_() for v in leaves]
    ref = [None if v is None else v.double().requires_grad_() for v in leaves]
    h, y = block_norms(*mine, scale=0.6, sigmoid=kind == "token")
    torch.autograd.backward([h, y], [wh, wy])
    hr, yr = plain_norms(torch, *ref, 0.6, kind == "token")
    torch.autograd.backward([hr, yr], [wh.double(), wy.double()])
    half = torch.finfo(t).eps / 2
    for a, b in zip(mine, ref):
        if a is None:
            continue
        assert a.grad.dtype == a.dtype and a.grad.shape == a.shape
        err = (a.grad.double() - b.grad).norm() / b.grad.norm()
        assert err.item() <= 4 * half + 2.0 ** -14, err.item()
    for a, b in ((h, hr), (y, yr)):
        assert ((a.double() - b).norm() / b.norm()).item() <= half + 2.0 ** -14


def test_norms_gradients_against_differences():
    """Central differences of the FP32 forward pass.  Against the gradient's projection they are off by the quotient's
    own error, which the FP64 formulas give, and by the outputs' roundings over 2 e: 20 u of each of the 2 x 192
    outputs (of size up to 5, under weights up to 5) in either loss, which is 384 * 25 * 20 u in all."""
    torch = gpuio.torch_cuda()
    from bit_microscaled_quantized_amd.blocks import block_norms
    H, e = 96, 2.0 ** -7
    leaves = [rnd(torch, 1, 2, H), rnd(torch, 2, 2, H), 1 + rnd(torch, 3, H, scale=0.2), 1 + rnd(torch, 4, H, scale=0.2),
              rnd(torch, 5, H)]
    wy, wh = rnd(torch, 6, 2, H).double(), rnd(torch, 7, 2, H).double()

    def loss(h, y):
        return h.double().mul(wh).sum() + y.double().mul(wy).sum()
    mine = [v.clone().requires_grad_() for v in leaves]
    loss(*block_norms(*mine, scale=0.6)).backward()
    ref = [v.double().requires_grad_() for v in leaves]
    loss(*plain_norms(torch, *ref, 0.6, False)).backward()
    for i in range(5):
        d = rnd(torch, 20 + i, *leaves[i].shape)
        d /= d.norm()
        up, down = list(leaves), list(leaves)
        up[i], down[i] = leaves[i] + e * d, leaves[i] - e * d
        width = (up[i].double() - down[i].double())  # 2 e d, as it was rounded
        slope = (loss(*block_norms(*up, scale=0.6)) - loss(*block_norms(*down, scale=0.6))).item()
        exact = (loss(*plain_norms(torch, *[v.double() for v in up], 0.6, False))
                 - loss(*plain_norms(torch, *[v.double() for v in down], 0.6, False))).item()
        own = abs(exact - ref[i].grad.mul(width).sum().item())
        want = mine[i].grad.double().mul(width).sum().item()
        assert abs(slope - want) <= own + 384 * 25 * 20 * U + 2.0 ** -16 * abs(want), (i, slope, want, own)


def kept(torch, v):
    from bit_microscaled_quantized_amd.blocks import keep8, restore8
    return restore8(*keep8(v.detach()), dtype=torch.float32)


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("act", ["none", "silu", "gelu", "relu2"])
@pytest.mark.parametrize("gated", [False, True])
def test_activation_gradients(dtype, act, gated):
    """Against FP64 autograd at the kept values, whose rounding is then no error of the gradient's."""
    torch = gpuio.torch_cuda()
    from bit_microscaled_quantized_amd.blocks import gated_act
    t = getattr(torch, dtype)
    wide = rnd(torch, 1, 4, 7, 400, dtype=t)
    gate = wide[..., :190].detach().requires_grad_()  # halves of a fused projection
    up = wide[..., 200:390].detach().requires_grad_() if gated else None
    dy = rnd(torch, 2, 4, 7, 190, dtype=t)
    y = gated_act(gate, up, act)
    y.backward(dy)
    half = torch.finfo(t).eps / 2
    plain = plain_act(torch, act, gate.detach().double()) * (up.detach().double() if gated else 1)
    assert ((y.double() - plain).norm() / plain.norm()).item() <= half + 2.0 ** -18
    ref = [kept(torch, v).double().requires_grad_() for v in (gate, up) if v is not None]
    out = plain_act(torch, act, ref[0]) * (ref[1] if gated else 1)
    out.backward(dy.double())
    for a, b in zip((gate, up), ref):
        assert ((a.grad.double() - b.grad).norm() / b.grad.norm()).item() <= half + 2.0 ** -18


def test_kept_values_are_near():
    torch = gpuio.torch_cuda()
    from bit_microscaled_quantized_amd.blocks import keep8, restore8
    for shape in ((5,), (3, 100), (2, 3, 64), (0, 8)):
        x = rnd(torch, 3, *shape)
        codes, scales = keep8(x)
        assert codes.shape == x.shape and scales.shape == (*shape[:-1], (shape[-1] + 31) // 32)
        y = restore8(codes, scales, torch.float32)
        # half a step of the block's scale, which is at most 2 / 127 of its largest magnitude
        assert x.numel() == 0 or bool(((y - x).abs() <= x.abs().max() / 127).all())
        assert restore8(codes, scales).dtype == torch.bfloat16


def test_activation_through_a_layer_that_keeps_no_activation():
    torch = gpuio.torch_cuda()
    from bit_microscaled_quantized_amd.blocks import gated_act, gated_act_linear
    gate, up = (rnd(torch, i, 3, 50, 160).requires_grad_() for i in (1, 2))
    w = rnd(torch, 3, 96, 160, scale=0.1).requires_grad_()
    dz = rnd(torch, 4, 3, 50, 96)
    z = gated_act_linear(gate, up, w, "silu")
    z.backward(dz)
    ref = [kept(torch, v).double().requires_grad_() for v in (gate, up)] + [w.detach().double().requires_grad_()]
    (plain_act(torch, "silu", ref[0]) * ref[1] @ ref[2].t()).backward(dz.double())
    for a, b in zip((gate, up, w), ref):
        # FP32 sums of 96, 96 and 150 products
        assert ((a.grad.double() - b.grad).norm() / b.grad.norm()).item() <= 200 * U + 2.0 ** -18
    assert torch.equal(z, torch.nn.functional.linear(gated_act(gate, up), w))
    # what is kept: no BF16 or FP32 activation
    saved = []
    with torch.autograd.graph.saved_tensors_hooks(lambda v: saved.append((tuple(v.shape), v.dtype)) or v, lambda v: v):
        gated_act_linear(gate.detach().bfloat16().requires_grad_(), up.detach().bfloat16(), w.detach().bfloat16())
    kinds = [d for s, d in saved if s != tuple(w.shape)]
    assert len(kinds) == 4 and set(kinds) == {torch.int8, torch.uint8}, saved


def block_step(torch, params, x, dtype):
    """One residual block in training: norms, gated activation, norms again."""
    from bit_microscaled_quantized_amd.blocks import block_norms, gated_act
    w_up, w_down, post, pre, gate_w = params
    h, y = block_norms(x, None, post, pre)
    u = torch.nn.functional.linear(y, w_up)
    a = gated_act(u[..., :u.shape[-1] // 2], u[..., u.shape[-1] // 2:], "silu")
    return block_norms(torch.nn.functional.linear(a, w_down), h, post, pre, torch.nn.functional.linear(y, gate_w),
                       scale=0.5, sigmoid=True)


def block_params(torch, H, F, dtype):
    return [rnd(torch, 1, 2 * F, H, scale=H ** -0.5).to(dtype).requires_grad_(),
            rnd(torch, 2, H, F, scale=F ** -0.5).to(dtype).requires_grad_(),
            (1 + rnd(torch, 3, H, scale=0.1)).to(dtype).requires_grad_(),
            (1 + rnd(torch, 4, H, scale=0.1)).to(dtype).requires_grad_(),
            rnd(torch, 5, H, H, scale=H ** -0.5).to(dtype).requires_grad_()]


def test_a_block_in_training():
    """A whole block in FP32 against FP64: the only roundings above FP32's are the kept inputs', half a step of at most
    2 / 127 of a block's largest value, which is at most 5 deviations here: errors of 0.04 / sqrt(3) deviations, which
    the activation's slopes (at most 1.1) pass on to the gradients relative to a factor of order one."""
    torch = gpuio.torch_cuda()
    H, F = 128, 320
    params = block_params(torch, H, F, torch.float32)
    x = rnd(torch, 9, 40, H).requires_grad_()
    h, y = block_step(torch, params, x, torch.float32)
    wh, wy = rnd(torch, 10, 40, H), rnd(torch, 11, 40, H)
    torch.autograd.backward([h, y], [wh, wy])
    ref = [p.detach().double().requires_grad_() for p in params]
    xr = x.detach().double().requires_grad_()
    h0, y0 = plain_norms(torch, xr, None, ref[2], ref[3], None, 1.0, False)
    u = y0 @ ref[0].t()
    a = plain_act(torch, "silu", u[:, :F]) * u[:, F:]
    hr, yr = plain_norms(torch, a @ ref[1].t(), h0, ref[2], ref[3], y0 @ ref[4].t(), 0.5, True)
    torch.autograd.backward([hr, yr], [wh.double(), wy.double()])
    assert ((h.double() - hr).norm() / hr.norm()).item() <= 2.0 ** -16
    assert ((y.double() - yr).norm() / yr.norm()).item() <= 2.0 ** -16
    for p, r in zip(params + [x], ref + [xr]):
        assert ((p.grad.double() - r.grad).norm() / r.grad.norm()).item() <= 0.04, p.shape


@pytest.mark.parametrize("T", [1, 5, 40, 200])
def test_a_block_in_serving(T):
    """norms -> 8-bit up-projection -> gated activation in 8 bits -> down-projection -> norms, against the same in FP64
    with the same 8-bit operands' roundings left out: each product's factors are off by half a step of 1 / 127 of
    their row's largest value, 4 to 5 deviations, so that a product is off by about 5 / 127 / sqrt(12) * sqrt(2) =
    1.6 % of its deviation, and two products, the activation between them (slopes up to 1.1 on both branches), add up
    to less than 6 %."""
    torch = gpuio.torch_cuda()
    from bit_microscaled_quantized_amd.blocks import Int8Linear, block_norms
    H, F = 256, 704
    params = [p.detach() for p in block_params(torch, H, F, torch.bfloat16)]
    up_g, up_u = Int8Linear(params[0][:F]), Int8Linear(params[0][F:])
    down = Int8Linear(params[1])
    x, r = rnd(torch, 9, T, H, dtype=torch.bfloat16), rnd(torch, 8, T, H, dtype=torch.bfloat16)
    with torch.no_grad():
        h, g = up_g.normed(x, r, params[2], params[3])
        h2, u = up_u.normed(x, r, params[2], params[3])
        z = down.gated(g, u)
        out_h, out_y = block_norms(z, h, params[2], params[3], scale=0.5)
    assert torch.equal(h, h2)
    d = [p.double() for p in params]
    hr, yr = plain_norms(torch, x.double(), r.double(), d[2], d[3], None, 1.0, False)
    a = plain_act(torch, "silu", yr @ d[0][:F].t()) * (yr @ d[0][F:].t())
    zr = a @ d[1].t()
    want_h, want_y = plain_norms(torch, zr, hr, d[2], d[3], None, 0.5, False)
    assert ((z.double() - zr).norm() / zr.norm()).item() <= 0.06
    assert ((out_h.double() - want_h).norm() / want_h.norm()).item() <= 0.06
    assert ((out_y.double() - want_y).norm() / want_y.norm()).item() <= 0.06
    # one token at a time gives the same, bit for bit: rows do not see each other
    with torch.no_grad():
        h1, g1 = up_g.normed(x[:1], r[:1], params[2], params[3])
        z1 = down.gated(g1, up_u.normed(x[:1], r[:1], params[2], params[3])[1])
    assert torch.equal(h1, h[:1]) and torch.equal(g1, g[:1]) and torch.equal(z1, z[:1])


def test_int8_linear_from_a_layer():
    torch = gpuio.torch_cuda()
    from bit_microscaled_quantized_amd.blocks import Int8Linear, int8_matmul, int8_quantize
    from bit_microscaled_quantized_amd.module import NVFP4Linear
    lin = NVFP4Linear(192, 320, seed=3)
    layer = Int8Linear.from_linear(lin)
    x = rnd(torch, 1, 2, 9, 192, dtype=torch.bfloat16)
    y = layer(x)
    assert y.shape == (2, 9, 320) and y.dtype == torch.bfloat16
    assert torch.equal(y.view(-1, 320), int8_matmul(*int8_quantize(x), layer.codes, layer.scales))
    want = x.double() @ lin.weight.detach().double().t()
    assert ((y.double() - want).norm() / want.norm()).item() <= 0.03  # 1.6 % as above, and BF16
    state = Int8Linear(torch.zeros(320, 192, device="cuda"))
    state.load_state_dict(layer.state_dict())
    assert torch.equal(state(x), y)
    # operands as slices of wider rows, aligned and not
    a, sa = int8_quantize(x)
    wide = torch.zeros((18, 400), dtype=torch.int8, device="cuda")
    for off in (0, 16, 5):
        wide[:, off:off + 192] = a
        assert torch.equal(int8_matmul(wide[:, off:off + 192], sa, layer.codes, layer.scales), y.view(-1, 320))
    with pytest.raises(RuntimeError, match="no gradient"):
        layer(x.clone().requires_grad_())
    with pytest.raises(ValueError, match="bias"):
        Int8Linear.from_linear(torch.nn.Linear(8, 8, device="cuda"))


def test_only_what_is_needed_is_computed():
    torch = gpuio.torch_cuda()
    from bit_microscaled_quantized_amd.blocks import BlockNorms, block_norms, gated_act
    H = 64
    x, g = rnd(torch, 1, 5, H), torch.ones(H, device="cuda")
    for i in range(5):
        leaves = [rnd(torch, 1, 5, H), rnd(torch, 2, 5, H), g.clone(), g.clone(), rnd(torch, 3, H)]
        leaves[i].requires_grad_()
        h, y = block_norms(*leaves)
        y.sum().backward()
        assert leaves[i].grad is not None and bool(torch.isfinite(leaves[i].grad).all())
    x = rnd(torch, 1, 5, H).requires_grad_()
    h, y = block_norms(x, None, g, g)
    h.square().sum().backward()  # y unused
    assert x.grad.norm().item() > 0
    u = rnd(torch, 2, 5, H).requires_grad_()
    gated_act(rnd(torch, 1, 5, H), u).sum().backward()
    assert u.grad.norm().item() > 0
    m = BlockNorms(H, layer_scale=0.1, dtype=torch.float32)
    h, y = m(x, x.detach())
    y.square().sum().backward()
    assert all(p.grad is not None for p in m.parameters())
    with pytest.raises(ValueError, match="gate"):
        m(x, None, gate=x)


def test_empty_batches():
    torch = gpuio.torch_cuda()
    from bit_microscaled_quantized_amd.blocks import Int8Linear, block_norms, gated_act, gated_act_linear
    g = torch.ones(32, device="cuda").requires_grad_()
    x = torch.empty(0, 3, 32, device="cuda").requires_grad_()
    gate = torch.ones(32, device="cuda").requires_grad_()
    h, y = block_norms(x, None, g, g, gate)
    (h.sum() + y.sum()).backward()
    assert x.grad.shape == x.shape and bool((g.grad == 0).all()) and bool((gate.grad == 0).all())
    u = torch.empty(0, 32, device="cuda").requires_grad_()
    w = torch.ones(8, 32, device="cuda").requires_grad_()
    gated_act(u).sum().backward()
    gated_act_linear(u, None, w).sum().backward()
    assert bool((w.grad == 0).all())
    assert Int8Linear(w)(u.detach()).shape == (0, 8)


@pytest.mark.parametrize("T", [1, 70, 300])
def test_captured_calls_replay_exactly(T):
    """Forward, backward and serving calls in one graph, replayed with other inputs and eager work between."""
    torch = gpuio.torch_cuda()
    import bit_microscaled_quantized_amd as nv
    from bit_microscaled_quantized_amd import blocks
    H, F = 192, 416
    params = [p.detach() for p in block_params(torch, H, F, torch.bfloat16)]
    up, down = blocks.Int8Linear(params[0][:F]), blocks.Int8Linear(params[1])
    x, r, dy = (rnd(torch, i, T, H, dtype=torch.bfloat16) for i in (6, 7, 8))
    gate = rnd(torch, 5, H, dtype=torch.bfloat16)

    def calls():
        with torch.no_grad():
            h, u = up.normed(x, r, params[2], params[3])
            z = down.gated(u, None, "relu2")
            codes, scales = blocks.keep8(z)
            y = blocks.restore8(codes, scales)
            stats = torch.ones(2, T, device="cuda")
            dx, dr = torch.empty_like(x), torch.empty_like(x)
            sums = [torch.empty(H, device="cuda") for _ in range(3)]
            ws = torch.empty(nv.nvfp4_block_norms_backward_workspace_size(T, H), dtype=torch.uint8, device="cuda")
            nv.nvfp4_block_norms_backward(dy, None, h, x, gate, 0, T, H, H, 0, H, H, 0, 1, params[2], params[3], 0, stats[0],
                                          stats[1], 0.5, dx, H, dr, H, sums[0], 0, sums[1], sums[2], ws)
        return [h, u, z, codes, scales, y, dx, dr, *sums]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        calls()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = calls()
    for i in range(4):
        for k, t in enumerate((x, r, dy)):
            t.copy_(rnd(torch, 100 * i + k, T, H, dtype=torch.bfloat16))
        want = [v.clone() for v in calls()]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want)), i


def test_two_streams_at_once():
    torch = gpuio.torch_cuda()
    from bit_microscaled_quantized_amd import blocks
    H, F, T = 512, 1408, 300
    params = [p.detach() for p in block_params(torch, H, F, torch.bfloat16)]
    up, down = blocks.Int8Linear(params[0][:F]), blocks.Int8Linear(params[1])
    xs = [rnd(torch, i, T, H, dtype=torch.bfloat16) for i in range(2)]

    def run(x):
        leaf = x.clone().requires_grad_()
        with torch.no_grad():
            h, u = up.normed(x, None, params[2], params[3])
            z = down.gated(u)
        a, b = blocks.block_norms(leaf, h, params[2], params[3])
        torch.autograd.backward([a, b], [z, z])
        return [h, u, z, a.detach(), b.detach(), leaf.grad]
    want = [[v.clone() for v in run(x)] for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(run(xs[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for r in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(r, want[i]))


def test_outputs_may_be_changed_in_place():
    torch = gpuio.torch_cuda()
    from bit_microscaled_quantized_amd.blocks import block_norms, gated_act
    g = torch.ones(64, device="cuda")
    x = rnd(torch, 1, 6, 64).requires_grad_()
    h, y = block_norms(x, None, g, g)
    y.mul_(2.0)
    y.sum().backward()
    first = x.grad.clone()
    x.grad = None
    (block_norms(x, None, g, g)[1] * 2.0).sum().backward()
    assert torch.equal(x.grad, first)
    gate = rnd(torch, 2, 6, 64).requires_grad_()
    a = gated_act(gate)
    a.add_(1.0)
    a.sum().backward()  # the codes are kept, not the output
    assert bool(torch.isfinite(gate.grad).all())


def test_arguments():
    torch = gpuio.torch_cuda()
    from bit_microscaled_quantized_amd import blocks
    x, g = rnd(torch, 1, 4, 64), torch.ones(64, device="cuda")
    bad = [lambda: blocks.block_norms(x, x[:2], g, g), lambda: blocks.block_norms(x, x.bfloat16(), g, g),
           lambda: blocks.block_norms(x, x, g[:32], g), lambda: blocks.block_norms(x, x, g, g.bfloat16()),
           lambda: blocks.block_norms(x, x, g, g, gate=x[:, :1]), lambda: blocks.block_norms(x, x, g, g, gate=x.bfloat16()),
           lambda: blocks.block_norms(x[:, :0], None, g[:0], g[:0]), lambda: blocks.block_norms(x[0, 0], None, g, g),
           lambda: blocks.gated_act(x, x[:2]), lambda: blocks.gated_act(x, x.bfloat16()),
           lambda: blocks.gated_act(x, None, "tanh"), lambda: blocks.gated_act(x[:, :0]),
           lambda: blocks.gated_act_linear(x, x, g[None, :32]), lambda: blocks.gated_act_linear(x, x, x.bfloat16()),
           lambda: blocks.restore8(x, g), lambda: blocks.int8_matmul(x, g, x, g),
           lambda: blocks.int8_matmul(x.to(torch.int8), g, x.to(torch.int8), g[:4]),
           lambda: blocks.int8_matmul(x.to(torch.int8)[:, :40], g[:4], x.to(torch.int8)[:, :40], g[:4]),
           lambda: blocks.Int8Linear(g), lambda: blocks.Int8Linear(x)(x[:, :32])]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    for call in (lambda: blocks.block_norms(x.half(), None, g.half(), g.half()), lambda: blocks.gated_act(x.half()),
                 lambda: blocks.keep8(x.double()), lambda: blocks.int8_quantize(x.half())):
        with pytest.raises(TypeError):
            call()
    with pytest.raises(blocks.nv.Nvfp4Error):
        blocks.block_norms(x, None, g, g, eps=-1.0)
