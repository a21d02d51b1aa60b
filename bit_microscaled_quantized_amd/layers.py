"""The operators between the quantized layers for PyTorch autograd, on the libnvfp4
kernels: dropout, the residual RMS norm and the linear cross entropy.

    y            = dropout(x, p, seed)
    h, y         = add_rms_norm(x, residual, gamma, eps, p, seed)   # y feeds the next layer, h the next addition
    codes, scales = rms_norm_mx8(x, residual, gamma, eps)           # inference: the norm in 8 bits
    loss         = linear_cross_entropy(x, weight, labels)           # mean over the labelled tokens

Nothing that can be formed again is saved: dropout's mask comes from its seed in
both directions, the norm keeps h and one number per row, the loss keeps one number
per token and neither logits nor probabilities.  Formulas and rounding are those of
include/nvfp4_layers.h.  BF16 and FP32 tensors (the loss BF16), any leading
dimensions; rows may be slices of a wider buffer.  Everything runs on torch's
current stream, on the current device, with buffers from its caching allocator.
"""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import nvfp4 as nv

_on_gpu = nv.on_current_device
_DT = {torch.bfloat16: nv.NVFP4_BF16, torch.float32: nv.NVFP4_F32}


def _dt(t) -> int:
    if t.dtype not in _DT:
        raise TypeError(f"expected a bfloat16 or float32 tensor, got {t.dtype}")
    return _DT[t.dtype]


def _norm_args(x, residual, gamma):
    """x and residual as matrices with their leading dimensions, and gamma packed."""
    _on_gpu(x, residual, gamma)
    if x.dim() == 0 or gamma.shape != x.shape[-1:]:
        raise ValueError(f"gamma must have the shape of x's last dimension, got {tuple(gamma.shape)} for "
                         f"{tuple(x.shape)}")
    if x.shape[-1] == 0:
        raise ValueError("expected at least one column")
    if residual is not None and (residual.shape != x.shape or residual.dtype != x.dtype):
        raise ValueError("residual must have x's shape and type")
    m, ld = _rows(x)
    r, ld_r = (None, 0) if residual is None else _rows(residual)
    return m, ld, r, ld_r, gamma.contiguous()


def _rows(t):
    """t as a matrix of its last dimension with unit stride (a copy only where that
    cannot be viewed), and its leading dimension.  A scalar is one element, and a tensor
    whose rows are empty has none."""
    cols = t.shape[-1] if t.dim() > 0 else 1
    m = t.reshape(-1, cols) if cols > 0 else t.reshape(0, 1)
    if m.stride(1) != 1 and m.shape[1] > 1 or m.stride(0) < m.shape[1] and m.shape[0] > 1:
        m = m.contiguous()
    return m, max(m.stride(0), m.shape[1])


def _operand(t):
    """_rows as the cross entropy takes them, 16-byte rows less than 2^22 elements apart:
    other slices are copied."""
    m, ld = _rows(t)
    if ld % 8 or ld >= 2 ** 22 or m.data_ptr() % 16:
        m, ld = m.clone(memory_format=torch.contiguous_format), m.shape[1]
    return m, ld


class _Dropout(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, p, seed):
        ctx.p, ctx.seed = p, seed
        return _run_dropout(x, p, seed)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        return _run_dropout(dy, ctx.p, ctx.seed), None, None


def _run_dropout(x, p, seed):
    _on_gpu(x)
    m, ld = _rows(x)
    y = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    nv.nvfp4_dropout(m, _dt(m), m.shape[0], m.shape[1], ld, p, seed, y, m.shape[1])
    return y


def dropout(x, p: float, seed: int):
    """Dropout of x with the mask of (seed, element index); the caller draws a new
    seed per use and step."""
    return _Dropout.apply(x, float(p), int(seed))


class _AddRmsNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, residual, gamma, eps, p, seed):
        m, ld, r, ld_r, g = _norm_args(x, residual, gamma)
        rows, cols = m.shape
        dt = _dt(m)
        # tensors of their own: y may be changed in place, and freed, while h is kept
        h = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        y = torch.empty_like(h)
        rstd = torch.empty(rows, dtype=torch.float32, device=m.device)
        nv.nvfp4_rms_norm(m, r, dt, rows, cols, ld, ld_r, g, _dt(g), eps, p, seed, h, cols, y, cols, None, None, rstd)
        ctx.set_materialize_grads(False)  # an unused h has no gradient to read
        ctx.save_for_backward(h, rstd, g)
        ctx.meta = (rows, cols, residual is not None, p, seed, gamma.dtype)
        return h, y

    @staticmethod
    @once_differentiable
    def backward(ctx, dh, dy):
        h, rstd, g = ctx.saved_tensors
        rows, cols, has_residual, p, seed, gamma_dtype = ctx.meta
        if dy is None and dh is None:
            return (None,) * 6
        dy, ld_dy = _rows(torch.zeros_like(h) if dy is None else dy)
        dh, ld_dh = (None, 0) if dh is None else _rows(dh)
        need_x, need_r, need_g = ctx.needs_input_grad[:3]
        need_r = need_r and has_residual
        if not (need_x or need_r or need_g):
            return (None,) * 6

        def out(need):
            return torch.empty_like(h) if need else None
        dx, dr = out(need_x), out(need_r)
        dg = torch.empty(cols, dtype=torch.float32, device=h.device) if need_g else None
        ws = None
        if need_g:
            ws = torch.empty(nv.nvfp4_rms_norm_backward_workspace_size(rows, cols), dtype=torch.uint8, device=h.device)
        nv.nvfp4_rms_norm_backward(dy, dh, h, _dt(h), rows, cols, ld_dy, ld_dh, cols, g, _dt(g), rstd, p, seed, dx,
                                   cols, dr, cols, dg, ws)
        return dx, dr, None if dg is None else dg.to(gamma_dtype), None, None, None


def add_rms_norm(x, residual, gamma, eps: float = 1e-5, p: float = 0.0, seed: int = 0):
    """(h, y): h = residual + dropout(x), y = h / sqrt(mean(h^2) + eps) * gamma;
    residual None is zero."""
    return _AddRmsNorm.apply(x, residual, gamma, float(eps), float(p), int(seed))


def rms_norm_mx8(x, residual, gamma, eps: float = 1e-5):
    """(h, codes, scales): the norm's output as E4M3 codes with one UE8M0 scale per 32
    columns (torch.float8_e4m3fn and torch.float8_e8m0fnu); no gradient."""
    m, ld, r, ld_r, g = _norm_args(x, residual, gamma)
    rows, cols = m.shape
    h = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    codes = torch.empty((rows, cols), dtype=torch.float8_e4m3fn, device=m.device)
    scales = torch.empty((rows, (cols + 31) // 32), dtype=torch.float8_e8m0fnu, device=m.device)
    nv.nvfp4_rms_norm(m, r, _dt(m), rows, cols, ld, ld_r, g, _dt(g), float(eps), 0.0, 0, h, cols, None, 0, codes, scales,
                      None)
    lead = x.shape[:-1]
    return h, codes.view(*lead, cols), scales.view(*lead, scales.shape[1])


class _LinearCrossEntropy(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, labels):
        if x.dtype != torch.bfloat16 or w.dtype != torch.bfloat16:
            raise TypeError("linear_cross_entropy takes bfloat16 hidden states and weight")
        _on_gpu(x, w, labels)
        if w.dim() != 2 or x.shape[-1:] != w.shape[1:] or labels.numel() * w.shape[1] != x.numel():
            raise ValueError("expected x [..., H], weight [V, H] and one label per token")
        lead, own = ([n for n in shape if n != 1] for shape in (x.shape[:-1], labels.shape))
        if lead != own and len(lead) > 1 and len(own) > 1:  # flat on either side, the order is plain
            raise ValueError(f"expected one label per token, got labels {tuple(labels.shape)} for x {tuple(x.shape)}")
        if w.shape[1] == 0:
            raise ValueError("expected at least one column")
        if labels.is_floating_point() or labels.is_complex():
            raise TypeError(f"expected integer labels, got {labels.dtype}")
        m, ld = _operand(x)
        wc, ld_w = _operand(w)
        T, H = m.shape
        V = w.shape[0]
        y = labels.reshape(-1).to(torch.int64).contiguous()
        loss = torch.empty(T, dtype=torch.float32, device=m.device)
        lse = torch.empty_like(loss)
        ws = torch.empty(nv.nvfp4_linear_cross_entropy_workspace_size(T, V, H, False), dtype=torch.uint8,
                         device=m.device)
        nv.nvfp4_linear_cross_entropy(T, V, H, m, ld, wc, ld_w, y, loss, lse, ws)
        ctx.save_for_backward(m, wc, y, lse)
        ctx.meta = (T, V, H, ld, ld_w, x.shape)
        return loss.view(labels.shape)

    @staticmethod
    @once_differentiable
    def backward(ctx, dloss):
        m, w, y, lse = ctx.saved_tensors
        T, V, H, ld, ld_w, shape = ctx.meta
        need_x, need_w = ctx.needs_input_grad[:2]
        if not (need_x or need_w):
            return None, None, None
        g = dloss.reshape(-1).float().contiguous()
        dx = torch.empty((T, H), dtype=torch.bfloat16, device=m.device) if need_x else None
        dw = torch.empty((V, H), dtype=torch.bfloat16, device=m.device) if need_w else None
        ws = torch.empty(nv.nvfp4_linear_cross_entropy_workspace_size(T, V, H, True), dtype=torch.uint8,
                         device=m.device)
        nv.nvfp4_linear_cross_entropy_backward(T, V, H, m, ld, w, ld_w, y, lse, g, dx, H, dw, nv.NVFP4_BF16, H, 0.0, ws)
        return None if dx is None else dx.view(shape), dw, None


def token_cross_entropy(x, w, labels):
    """Loss of each token (0 where its label is outside [0, V)), FP32.  labels have x's
    leading dimensions, or are flat in their order; the loss has the labels' shape."""
    return _LinearCrossEntropy.apply(x, w, labels)


def linear_cross_entropy(x, w, labels):
    """Mean loss of the tokens whose label lies in [0, V); 0 if there are none."""
    valid = (labels >= 0) & (labels < w.shape[0])
    return token_cross_entropy(x, w, labels).sum() / valid.sum().clamp(min=1)


def _capturing(x) -> bool:
    return x.is_cuda and torch.cuda.is_current_stream_capturing()


class AddRMSNorm(torch.nn.Module):
    """add_rms_norm with its gain.  In training, dropout takes a new mask every call: its
    seed is a draw from torch's CPU generator, mixed with the module's seed (for modules,
    or ranks, whose generators run alike).  So torch.manual_seed repeats a run's masks,
    the generator's saved state resumes them, and torch.utils.checkpoint, which restores
    that state, recomputes a forward pass with the mask it had.  A launch's seed is its
    argument, so every replay of a captured graph would drop the same elements: under
    capture dropout is refused."""

    def __init__(self, features: int, eps: float = 1e-5, p: float = 0.0, seed: int = 0, device="cuda", dtype=None):
        super().__init__()
        self.gamma = torch.nn.Parameter(torch.ones(features, device=device, dtype=dtype or torch.bfloat16))
        self.eps, self.p, self.seed = eps, p, seed

    def forward(self, x, residual=None):
        if not self.training or self.p == 0.0:
            return add_rms_norm(x, residual, self.gamma, self.eps)
        if _capturing(x):
            raise RuntimeError("AddRMSNorm draws a new dropout mask every call, and a captured graph would replay "
                               "one: capture it with p = 0, or add_rms_norm with a seed of your own")
        draw = int(torch.randint(2 ** 63 - 1, (), dtype=torch.int64, device="cpu"))
        # an odd factor: different seeds below 2^64 stay different
        s = (draw ^ self.seed * 0x9E3779B97F4A7C15) & (2 ** 64 - 1)
        return add_rms_norm(x, residual, self.gamma, self.eps, self.p, s)
