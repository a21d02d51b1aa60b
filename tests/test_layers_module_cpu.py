"""The autograd layer's own arithmetic on the host: a stand-in written in elementary torch
operations takes the place of the kernels, so that seeds, shapes and refusals of
bit_microscaled_quantized_amd.layers are tested without a device."""
import copy

import pytest
import torch
from torch.utils.checkpoint import checkpoint

from bit_microscaled_quantized_amd import layers

COLS = 48


def _mask(rows, cols, p, seed):
    g = torch.Generator().manual_seed(seed % 2 ** 63)
    return (torch.rand(rows, cols, generator=g) >= p) / (1.0 - p)


class Kernels:
    """nvfp4_rms_norm and its backward for packed FP32 host tensors; keeps the seeds it was given."""

    def __init__(self):
        self.seeds = []

    def nvfp4_rms_norm(self, x, r, dt, rows, cols, ld_x, ld_r, gamma, gdt, eps, p, seed, h, ld_h, y, ld_y, codes, scales,
                       rstd):
        self.seeds.append(seed % 2 ** 64)
        h.copy_((x * _mask(rows, cols, p, seed) + (0 if r is None else r)).view(h.shape))
        rstd.copy_(torch.rsqrt(h.view(rows, cols).square().mean(1) + eps))
        y.copy_((h.view(rows, cols) * rstd[:, None] * gamma).view(y.shape))

    def nvfp4_rms_norm_backward_workspace_size(self, rows, cols):
        return 0

    def nvfp4_rms_norm_backward(self, dy, dh, h, dt, rows, cols, ld_dy, ld_dh, ld_h, gamma, gdt, rstd, p, seed, dx, ld_dx,
                                dr, ld_dr, dgamma, ws):
        n = h.view(rows, cols) * rstd[:, None]
        gy = dy.view(rows, cols) * gamma
        g = rstd[:, None] * (gy - n * (gy * n).mean(1, keepdim=True)) + (0 if dh is None else dh.view(rows, cols))
        for out, v in ((dx, g * _mask(rows, cols, p, seed)), (dr, g)):
            if out is not None:
                out.copy_(v.view(out.shape))
        if dgamma is not None:
            dgamma.copy_((dy.view(rows, cols) * n).sum(0))


@pytest.fixture
def kernels(monkeypatch):
    k = Kernels()
    for name in ("nvfp4_rms_norm", "nvfp4_rms_norm_backward", "nvfp4_rms_norm_backward_workspace_size"):
        monkeypatch.setattr(layers.nv, name, getattr(k, name))
    monkeypatch.setattr(layers, "_on_gpu", lambda *tensors: None)
    return k


def norm(**kw):
    return layers.AddRMSNorm(COLS, p=0.5, device="cpu", dtype=torch.float32, **kw)


def branch(module, x, r):
    h, y = module(torch.tanh(x), r)
    return (h * 0.3 + y.square()).sum()


@pytest.mark.parametrize("use_reentrant", [False, True])
def test_checkpointed_norm_repeats_its_mask(kernels, use_reentrant):
    """The recomputed forward has to draw the mask of the first one: gradients are those
    without checkpointing, bit for bit."""
    module = norm(seed=3)
    g = torch.Generator().manual_seed(1)
    data = [torch.randn(6, COLS, generator=g) for _ in range(2)]
    grads = []
    for through in (lambda f, *a: f(*a), lambda f, *a: checkpoint(f, *a, use_reentrant=use_reentrant)):
        torch.manual_seed(7)
        x, r = (t.clone().requires_grad_() for t in data)
        m = copy.deepcopy(module)
        through(lambda a, b: branch(m, a, b), x, r).backward()
        grads.append((x.grad, r.grad, m.gamma.grad))
    assert all(torch.equal(a, b) for a, b in zip(*grads))
    assert len(kernels.seeds) == 3 and len(set(kernels.seeds)) == 1


def test_every_norm_and_call_has_a_mask_of_its_own(kernels):
    """Modules built alike, and the calls of one module, drop different elements; modules
    that differ in their seed do too where torch's generator stands at the same state."""
    x = torch.randn(2, COLS)
    a, b = norm(), norm()
    for _ in range(3):
        for m in (a, b):
            m(x)
    torch.manual_seed(5)
    norm(seed=1)(x)
    torch.manual_seed(5)
    norm(seed=2)(x)
    assert len(set(kernels.seeds)) == 8, kernels.seeds


def test_a_resumed_run_continues_its_masks(kernels):
    """The parameters and torch's generator state, saved and restored, are all it takes."""
    x = torch.randn(2, COLS)
    torch.manual_seed(11)
    m = norm(seed=4)
    m(x)
    saved, rng = copy.deepcopy(m.state_dict()), torch.get_rng_state()
    m(x)
    other = norm(seed=4)
    other.load_state_dict(saved)
    torch.manual_seed(0)
    torch.set_rng_state(rng)
    other(x)
    assert kernels.seeds[2] == kernels.seeds[1] != kernels.seeds[0]


def test_evaluation_draws_nothing(kernels):
    m = norm(seed=1).eval()
    rng = torch.get_rng_state()
    h, _ = m(torch.ones(2, COLS))
    assert torch.equal(h, torch.ones(2, COLS)) and torch.equal(torch.get_rng_state(), rng)


def test_a_captured_call_would_repeat_one_mask_and_is_refused(kernels, monkeypatch):
    """A launch's seed is its argument: every replay would drop what the capture dropped.
    Without dropout, and with a seed that the caller gives, there is nothing to refuse."""
    monkeypatch.setattr(layers, "_capturing", lambda x: True)
    m, x = norm(seed=1), torch.ones(2, COLS)
    with pytest.raises(RuntimeError, match="capture"):
        m(x)
    assert kernels.seeds == []
    layers.add_rms_norm(x, None, m.gamma, p=0.5, seed=9)
    m.eval()(x)
    assert kernels.seeds == [9, 0]


class OnDevice:
    """What the device checks look at of a tensor on GPU `index`."""
    is_cuda = True

    def __init__(self, index):
        self.device = torch.device("cuda", index)


def test_tensors_on_another_device_than_the_current_one_are_refused(monkeypatch):
    """The kernels are launched on the current device, on its stream."""
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    layers._on_gpu(OnDevice(0), OnDevice(0), None)
    for tensors in ((OnDevice(1),), (OnDevice(1), OnDevice(1)), (OnDevice(0), OnDevice(1))):
        with pytest.raises(ValueError, match="cuda:"):
            layers._on_gpu(*tensors)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    layers._on_gpu(OnDevice(1), OnDevice(1))


class LossKernels:
    """Keeps the leading dimensions that the cross entropy was given, and refuses those that
    the library refuses."""

    def __init__(self):
        self.lds = []

    def workspace_size(self, T, V, H, train):
        return 0

    def forward(self, T, V, H, x, ld_x, w, ld_w, labels, loss, lse, ws):
        self.lds.append((ld_x, ld_w))
        for t, rows, ld in ((x, T, ld_x), (w, V, ld_w)):
            assert H <= ld < 2 ** 22 and ld % 8 == 0 and t.data_ptr() % 16 == 0
            assert rows <= 1 or ld == t.stride(0)
        z = x.double() @ w.double().t()
        lse.copy_(torch.logsumexp(z, 1))
        ok = (labels >= 0) & (labels < V)
        loss.copy_(torch.where(ok, lse - z.gather(1, labels.clamp(0, V - 1)[:, None])[:, 0], 0.0))


@pytest.fixture
def loss_kernels(monkeypatch):
    k = LossKernels()
    monkeypatch.setattr(layers.nv, "nvfp4_linear_cross_entropy", k.forward)
    monkeypatch.setattr(layers.nv, "nvfp4_linear_cross_entropy_workspace_size", k.workspace_size)
    monkeypatch.setattr(layers, "_on_gpu", lambda *tensors: None)
    return k


@pytest.mark.parametrize("batch,seq", [(1, 2 ** 16 + 8), (3, 2 ** 16 + 8), (1, 50), (3, 50)])
def test_loss_of_the_last_tokens_of_long_sequences(loss_kernels, batch, seq):
    """hidden[:, -1]: rows a whole sequence apart, further than the kernels' leading
    dimension goes (2^22) for the long ones; one row has no distance at all."""
    H = 64
    hidden = torch.randn(1, 1, H).bfloat16().expand(batch, seq, H).contiguous()
    hidden[:, -1] = torch.randn(batch, H).bfloat16()
    w = torch.randn(40, H).bfloat16()
    y = torch.arange(batch)
    got = layers.token_cross_entropy(hidden[:, -1], w, y)
    want = layers.token_cross_entropy(hidden[:, -1].clone(), w, y)
    assert torch.equal(got, want) and got.shape == (batch,)
    # a slice is read where it lies, where it can be
    assert loss_kernels.lds[0][0] == (64 if batch == 1 or seq * H >= 2 ** 22 else seq * H)


@pytest.mark.parametrize("off", [1, 4, 8])
def test_loss_of_packed_rows_that_start_anywhere(loss_kernels, off):
    """Rows that lie packed but not on 16 bytes (a slice of a flat buffer) are copied too."""
    H, T, V = 64, 5, 40
    x = torch.randn(T * H + off).bfloat16()[off:].view(T, H)
    w = torch.randn(V * H + off).bfloat16()[off:].view(V, H)
    y = torch.arange(T)
    got = layers.token_cross_entropy(x, w, y)
    want = layers.token_cross_entropy(x.clone(), w.clone(), y)
    assert torch.equal(got, want)


@pytest.mark.parametrize("lead", [(0,), (3, 0), (0, 5), (2, 3), ()])
def test_eight_bit_norm_of_any_leading_dimensions(monkeypatch, lead):
    """An empty batch gives empty outputs of its shape."""
    monkeypatch.setattr(layers.nv, "nvfp4_rms_norm", lambda *a: None)
    monkeypatch.setattr(layers, "_on_gpu", lambda *tensors: None)
    x = torch.ones(*lead, 72).bfloat16()
    h, codes, scales = layers.rms_norm_mx8(x, x, torch.ones(72))
    assert h.shape == x.shape and codes.shape == (*lead, 72) and scales.shape == (*lead, 3)
    assert codes.dtype == torch.float8_e4m3fn and scales.dtype == torch.float8_e8m0fnu


@pytest.mark.parametrize("shape", [(), (1,), (0,), (3, 0), (0, 4), (2, 3, 4)])
def test_dropout_of_any_shape(monkeypatch, shape):
    """Scalars and empty tensors included, in both directions; the library sees a matrix
    that its checks take."""
    calls = []

    def dropout(x, dt, rows, cols, ld_x, p, seed, y, ld_y):
        assert rows >= 0 and cols >= 1 and ld_x >= cols and ld_y >= cols and x.shape == (rows, cols)
        calls.append(rows * cols)
        y.copy_(x.view(y.shape) * 2)
    monkeypatch.setattr(layers.nv, "nvfp4_dropout", dropout)
    monkeypatch.setattr(layers, "_on_gpu", lambda *tensors: None)
    x = torch.randn(shape, requires_grad=True)
    y = layers.dropout(x, 0.5, 3)
    y.sum().backward()
    assert torch.equal(y, 2 * x) and x.grad.shape == x.shape and bool((x.grad == 2).all())
    assert calls == [x.numel()] * 2
    with pytest.raises(TypeError):
        layers.dropout(torch.ones(shape, dtype=torch.float16), 0.5, 3)


def test_rows_without_columns_are_refused(monkeypatch):
    """A norm or a product over nothing has no value."""
    monkeypatch.setattr(layers, "_on_gpu", lambda *tensors: None)
    x, w, y = torch.empty(3, 0).bfloat16(), torch.empty(7, 0).bfloat16(), torch.zeros(3, dtype=torch.int64)
    for norm_of in (layers.add_rms_norm, layers.rms_norm_mx8):
        with pytest.raises(ValueError, match="column"):
            norm_of(x, None, torch.empty(0))
    with pytest.raises(ValueError, match="column"):
        layers.token_cross_entropy(x, w, y)


def test_labels_belong_to_their_tokens(loss_kernels):
    """Labels of the tokens' own shape, or flat, in their order; transposed ones, as many
    as there are tokens, would score every token by another's label."""
    x, w = torch.randn(2, 3, 64).bfloat16(), torch.randn(10, 64).bfloat16()
    y = torch.arange(6).view(2, 3)
    want = layers.token_cross_entropy(x, w, y)
    assert want.shape == (2, 3)
    for same in (y.view(6), y[..., None], y[None]):
        assert torch.equal(layers.token_cross_entropy(x, w, same).view(2, 3), want)
    assert torch.equal(layers.token_cross_entropy(x.view(6, 64), w, y), want)
    for wrong in (y.t(), y.view(1, 3, 2), y.view(3, 2)):
        with pytest.raises(ValueError, match="label"):
            layers.token_cross_entropy(x, w, wrong)
