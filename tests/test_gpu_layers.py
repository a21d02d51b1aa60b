"""The autograd layer over the operators between the quantized layers, their use
together, under graph capture and on two streams."""
import os
import sys

import pytest

from tests import gpuio

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def plain_step(torch, x, r, gamma, w, labels, eps=1e-5):
    """FP64 loss of norm and head, for autograd."""
    h = r + x
    y = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + eps) * gamma
    z = y.reshape(-1, y.shape[-1]) @ w.t()
    valid = (labels >= 0) & (labels < w.shape[0])
    picked = z.gather(1, torch.where(valid, labels, 0).reshape(-1, 1))[:, 0]
    loss = torch.where(valid.reshape(-1), torch.logsumexp(z, 1) - picked, 0.0)
    return loss.sum() / valid.sum().clamp(min=1), h


def test_gradients_through_norm_and_loss():
    """x -> add_rms_norm -> linear_cross_entropy against FP64 autograd of the same
    formulas.  y, d, dy and the gradients are each rounded to BF16 once (2^-8 of the
    value): a dozen such roundings, added as norms, stay within 2^-5."""
    torch = gpuio.torch_cuda()
    from bit_microscaled_quantized_amd.layers import add_rms_norm, linear_cross_entropy
    g = torch.Generator(device="cuda").manual_seed(3)
    B, S, H, V = 3, 50, 256, 777
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")
    leaves = [rnd(B, S, H).bfloat16(), rnd(B, S, H).bfloat16(), (1 + 0.2 * rnd(H)).bfloat16(),
              (rnd(V, H) * 0.06).bfloat16()]
    labels = torch.randint(V, (B, S), generator=g, device="cuda")
    labels[0, ::3] = -100
    mine = [t.clone().requires_grad_() for t in leaves]
    h, y = add_rms_norm(mine[0], mine[1], mine[2])
    loss = linear_cross_entropy(y, mine[3], labels) + h.float().square().mean() * 0.01
    loss.backward()
    ref = [t.double().requires_grad_() for t in leaves]
    want, hr = plain_step(torch, *ref, labels)
    want = want + hr.square().mean() * 0.01
    want.backward()
    assert abs(loss.item() - want.item()) <= 2.0 ** -8 * want.item()
    for a, b in zip(mine, ref):
        err = (a.grad.double() - b.grad).norm() / b.grad.norm()
        assert err.item() <= 2.0 ** -5, err.item()


def test_dropout_backward_repeats_the_mask():
    torch = gpuio.torch_cuda()
    from bit_microscaled_quantized_amd.layers import add_rms_norm, dropout
    x = torch.randn(7, 33, device="cuda", requires_grad=True)
    y = dropout(x, 0.4, 5)
    y.backward(torch.ones_like(y))
    assert torch.equal(x.grad != 0, y != 0)
    wide = torch.randn(5, 3, 64, device="cuda")[..., 5:38].requires_grad_()  # a slice of wider rows
    h, _ = add_rms_norm(wide, None, torch.ones(33, device="cuda"), p=0.4, seed=9)
    (g,) = torch.autograd.grad(h.sum(), wide)
    assert g.shape == wide.shape and torch.equal(g != 0, h != 0)


def test_only_what_is_needed_is_computed():
    torch = gpuio.torch_cuda()
    from bit_microscaled_quantized_amd.layers import add_rms_norm, token_cross_entropy
    x = torch.randn(4, 64, device="cuda").bfloat16()
    gamma = torch.ones(64, device="cuda", requires_grad=True)
    h, y = add_rms_norm(x, None, gamma)
    y.sum().backward()
    assert gamma.grad is not None
    w = torch.randn(50, 64, device="cuda").bfloat16().requires_grad_()
    token_cross_entropy(x, w, torch.zeros(4, dtype=torch.int64, device="cuda")).sum().backward()
    assert w.grad is not None and w.grad.isfinite().all()


def test_arguments_of_the_autograd_layer():
    """What does not fit is refused before any kernel runs, host tensors beside device ones too."""
    torch = gpuio.torch_cuda()
    from bit_microscaled_quantized_amd import layers
    x = torch.ones(4, 64, device="cuda").bfloat16()
    g, w = torch.ones(64, device="cuda"), torch.ones(10, 64, device="cuda").bfloat16()
    y = torch.zeros(4, dtype=torch.int64, device="cuda")
    for norm in (layers.add_rms_norm, layers.rms_norm_mx8):
        for r, gain in ((x[:3], g), (x.float(), g), (x, g[:32]), (x, g[None]), (x.cpu(), g), (x, g.cpu())):
            with pytest.raises(ValueError):
                norm(x, r, gain)
        with pytest.raises(TypeError):
            norm(x.half(), None, g)
    for args in ((x, w[:, :32], y), (x, w, y[:3]), (x, w, y.cpu()), (x, w.cpu(), y), (x, w[0], y)):
        with pytest.raises(ValueError):
            layers.token_cross_entropy(*args)
    for args in ((x.float(), w, y), (x, w.float(), y), (x, w, y.float())):
        with pytest.raises(TypeError):
            layers.token_cross_entropy(*args)
    with pytest.raises(TypeError):
        layers.dropout(y, 0.1, 1)


def test_outputs_may_be_changed_in_place():
    """y may be, since only h is kept for the gradient; a change of h is reported."""
    torch = gpuio.torch_cuda()
    from bit_microscaled_quantized_amd.layers import add_rms_norm
    x = torch.randn(3, 5, 96, device="cuda", requires_grad=True)
    gamma = torch.ones(96, device="cuda", requires_grad=True)
    h, y = add_rms_norm(x, None, gamma)
    (y * 2.0).sum().backward()
    want = x.grad.clone()
    x.grad = None
    h, y = add_rms_norm(x, None, gamma)
    y.mul_(2.0).sum().backward()
    assert torch.equal(x.grad, want) and torch.isfinite(want).all()
    h, y = add_rms_norm(x, None, gamma)
    h.mul_(2.0)
    with pytest.raises(RuntimeError):
        y.sum().backward()


def test_example_trains():
    import train_ffn_head
    losses, diff = train_ffn_head.train(steps=25, hidden=256, ffn=512, blocks=2, vocab=2048, tokens=1024, report=None)
    assert losses[-1] < 0.7 * losses[0], losses
    assert diff <= 2.0 ** -3  # half a step of E4M3 on both sides of a BF16 value, relative to the largest


def _calls(torch, nv, b, seed):
    """Every entry point once; BF16, H = 264, T = 130."""
    T, V, H = b["T"], b["V"], b["H"]
    bf = nv.NVFP4_BF16
    nv.nvfp4_dropout(b["x"], bf, T, H, H, 0.2, seed, b["y0"], H)
    nv.nvfp4_rms_norm(b["y0"], b["r"], bf, T, H, H, H, b["g"], bf, 1e-5, 0.1, seed + 1, b["h"], H, b["y"], H, None, None,
                      b["rstd"])
    nv.nvfp4_rms_norm(b["y0"], b["r"], bf, T, H, H, H, b["g"], bf, 1e-5, 0.0, 0, None, 0, None, 0, b["codes"],
                      b["scales"], None)
    nv.nvfp4_linear_cross_entropy(T, V, H, b["y"], H, b["w"], H, b["labels"], b["loss"], b["lse"], b["ws"])
    nv.nvfp4_linear_cross_entropy_backward(T, V, H, b["y"], H, b["w"], H, b["labels"], b["lse"], b["dloss"], b["dy"], H,
                                           b["dw"], bf, H, 0.0, b["ws"])
    nv.nvfp4_rms_norm_backward(b["dy"], None, b["h"], bf, T, H, H, 0, H, b["g"], bf, b["rstd"], 0.1, seed + 1, b["dx"], H,
                               b["dr"], H, b["dg"], b["wsn"])


OUT = ("y0", "h", "y", "rstd", "codes", "scales", "loss", "lse", "dy", "dw", "dx", "dr", "dg")


def _buffers(torch, nv, T=130, V=1000, H=264, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")
    e = lambda *s, t=torch.bfloat16: torch.empty(s, dtype=t, device="cuda")
    labels = torch.randint(V, (T,), generator=g, device="cuda")
    labels[::5] = -100
    b = dict(T=T, V=V, H=H, x=rnd(T, H).bfloat16(), r=rnd(T, H).bfloat16(), g=(1 + 0.1 * rnd(H)).bfloat16(),
             w=(rnd(V, H) * 0.05).bfloat16(), labels=labels, dloss=rnd(T) / T)
    b.update(y0=e(T, H), h=e(T, H), y=e(T, H), rstd=e(T, t=torch.float32), codes=e(T, H, t=torch.uint8),
             scales=e(T, (H + 31) // 32, t=torch.uint8), loss=e(T, t=torch.float32), lse=e(T, t=torch.float32),
             dy=e(T, H), dw=e(V, H), dx=e(T, H), dr=e(T, H), dg=e(H, t=torch.float32),
             ws=e(nv.nvfp4_linear_cross_entropy_workspace_size(T, V, H, True), t=torch.uint8),
             wsn=e(nv.nvfp4_rms_norm_backward_workspace_size(T, H), t=torch.uint8))
    return b


def _same(torch, a, b, what):
    for k in OUT:
        assert torch.equal(a[k].view(torch.uint8), b[k].view(torch.uint8)), f"{what}: {k} differs"


@pytest.mark.parametrize("T", [3, 130, 300])
def test_captured_calls_replay_exactly(T):
    """All entry points in one graph, replayed three times with eager calls and
    overwritten outputs between: every replay gives the eager results' bytes."""
    torch = gpuio.torch_cuda()
    import bit_microscaled_quantized_amd as nv
    eager, graph = _buffers(torch, nv, T), _buffers(torch, nv, T)
    _calls(torch, nv, eager, 5)
    want = {k: eager[k].clone() for k in OUT}
    g = torch.cuda.CUDAGraph()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        with torch.cuda.graph(g, stream=stream):
            _calls(torch, nv, graph, 5)
    for rep in range(3):
        for k in OUT + ("ws", "wsn"):
            graph[k].view(torch.uint8).fill_(0x5A)
        _calls(torch, nv, eager, 5)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        _same(torch, graph, want, f"replay {rep}")
        _same(torch, eager, want, f"eager calls before replay {rep}")


def test_two_streams_at_once():
    """Two streams with their own buffers, interleaved: the results of one at a time."""
    torch = gpuio.torch_cuda()
    import bit_microscaled_quantized_amd as nv
    one, two = _buffers(torch, nv, seed=1), _buffers(torch, nv, seed=2)
    _calls(torch, nv, one, 7)
    _calls(torch, nv, two, 8)
    want = [{k: b[k].clone() for k in OUT} for b in (one, two)]
    for b in (one, two):
        for k in OUT:
            b[k].view(torch.uint8).fill_(0x5A)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(10):
        for s, b, seed in zip(streams, (one, two), (7, 8)):
            with torch.cuda.stream(s):
                _calls(torch, nv, b, seed)
    torch.cuda.synchronize()
    for b, w, name in zip((one, two), want, "ab"):
        _same(torch, b, w, f"stream {name}")


@pytest.mark.parametrize("use_reentrant", [False, True])
def test_checkpointed_norm_with_dropout(use_reentrant):
    """Activation checkpointing gives the bytes of the step without it, dropout's mask included."""
    torch = gpuio.torch_cuda()
    from torch.utils.checkpoint import checkpoint
    from bit_microscaled_quantized_amd.layers import AddRMSNorm
    g = torch.Generator(device="cuda").manual_seed(4)
    data = [torch.randn(40, 264, generator=g, device="cuda").bfloat16() for _ in range(2)]
    module = AddRMSNorm(264, p=0.3, seed=1)

    def branch(a, b):
        h, y = module(torch.tanh(a), b)
        return h.float().sum() + y.float().square().sum()
    grads = []
    for through in (lambda f, *a: f(*a), lambda f, *a: checkpoint(f, *a, use_reentrant=use_reentrant)):
        torch.manual_seed(7)
        module.zero_grad()
        x, r = (t.clone().requires_grad_() for t in data)
        through(branch, x, r).backward()
        grads.append((x.grad, r.grad, module.gamma.grad.clone()))
    assert all(torch.equal(a, b) for a, b in zip(*grads))
    dropped = grads[0][0] == 0
    assert 0.2 < float(dropped.float().mean()) < 0.4


def test_captured_module_refuses_dropout():
    """A graph would replay one mask; p = 0 and a seed of the caller's are captured."""
    torch = gpuio.torch_cuda()
    from bit_microscaled_quantized_amd.layers import AddRMSNorm, add_rms_norm
    x = torch.randn(3, 64, device="cuda").bfloat16()
    module = AddRMSNorm(64, p=0.3)
    with torch.no_grad():
        want = add_rms_norm(x, None, module.gamma, p=0.3, seed=5)[1]
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            with pytest.raises(RuntimeError, match="captured graph"):
                module(x)
            got = add_rms_norm(x, None, module.gamma, p=0.3, seed=5)[1]
            kept = module.eval()(x)[0]
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, want) and torch.equal(kept, x)


def test_loss_of_the_last_tokens_of_long_sequences():
    """Hidden states a whole sequence apart, more than 2^22 elements: value and gradient of
    the packed rows."""
    torch = gpuio.torch_cuda()
    from bit_microscaled_quantized_amd.layers import linear_cross_entropy
    g = torch.Generator(device="cuda").manual_seed(6)
    hidden = torch.randn(3, 2100, 2048, generator=g, device="cuda").bfloat16().requires_grad_()
    w = (torch.randn(300, 2048, generator=g, device="cuda") * 0.02).bfloat16()
    y = torch.tensor([5, 299, -100], device="cuda")
    packed = hidden.detach()[:, -1].clone().requires_grad_()
    linear_cross_entropy(hidden[:, -1], w, y).backward()
    linear_cross_entropy(packed, w, y).backward()
    assert torch.equal(hidden.grad[:, -1], packed.grad) and bool((packed.grad[:2] != 0).any())
    assert bool((hidden.grad[:, :-1] == 0).all())


def test_empty_batches():
    """No rows, no tokens: empty outputs of the shape, zero gradients of what they share."""
    torch = gpuio.torch_cuda()
    from bit_microscaled_quantized_amd import layers
    x = torch.empty(2, 0, 64, device="cuda", dtype=torch.bfloat16, requires_grad=True)
    gamma = torch.ones(64, device="cuda", requires_grad=True)
    w = torch.ones(10, 64, device="cuda", dtype=torch.bfloat16, requires_grad=True)
    h, y = layers.add_rms_norm(layers.dropout(x, 0.5, 1), x, gamma)
    loss = layers.linear_cross_entropy(y, w, torch.empty(2, 0, dtype=torch.int64, device="cuda"))
    (loss + h.float().sum()).backward()
    assert float(loss.detach()) == 0 and y.shape == x.grad.shape == x.shape
    assert bool((gamma.grad == 0).all()) and bool((w.grad == 0).all())
    _, codes, scales = layers.rms_norm_mx8(x.detach(), None, gamma.detach())
    assert codes.shape == (2, 0, 64) and scales.shape == (2, 0, 2)


def test_dropout_of_scalars_and_empty_rows():
    torch = gpuio.torch_cuda()
    from bit_microscaled_quantized_amd.layers import dropout
    for shape in ((), (1,), (3, 0), (0, 4)):
        x = torch.ones(shape, device="cuda", requires_grad=True)
        y = dropout(x, 0.25, 6)
        y.sum().backward()
        assert y.shape == x.grad.shape == x.shape and torch.equal(x.grad, y)
        assert bool(((y == 0) | ((y - 4 / 3).abs() < 1e-6)).all())
