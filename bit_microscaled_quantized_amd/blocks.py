"""The operators of a residual block in eight bits for PyTorch, on the libnvfp4 kernels:
the norms around a block with its gate and residual scale, the gated activation whose
inputs are kept in 8 bits, and the product of 8-bit integers for serving.

    h, y = block_norms(x, residual, post_gamma, pre_gamma, gate, scale)   # x: a block's output; y: the next one's input
    a    = gated_act(gate, up, "silu")                # act(gate) * up; both kept in 8 bits for the backward pass
    z    = gated_act_linear(gate, up, weight)         # that through a BF16 linear layer, without keeping a
    codes, scales = keep8(x);  x2 = restore8(codes, scales, x.dtype)      # any tensor in 8 bits

    layer = Int8Linear.from_linear(linear)            # inference: 8-bit weight, 8-bit input per token
    y = layer(x);  y = layer.gated(gate, up, "silu");  h, y = layer.normed(x, residual, post_gamma, pre_gamma)

Formulas, roundings and formats are those of include/nvfp4_blocks.h.  BF16 and FP32
tensors, any leading dimensions; rows may be slices of a wider buffer.  Everything runs
on torch's current stream, on the current device, with buffers from its caching
allocator.  A backward pass is captured into a graph through torch.autograd.grad, or while
no eager graph of the same leaves lives.
"""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import nvfp4 as nv
from .layers import _dt, _on_gpu, _rows

_ACTS = {"none": nv.NVFP4_ACT_NONE, "silu": nv.NVFP4_ACT_SILU, "gelu": nv.NVFP4_ACT_GELU, "relu2": nv.NVFP4_ACT_RELU2}


def _act_code(act: str) -> int:
    if act not in _ACTS:
        raise ValueError(f"act must be one of {', '.join(_ACTS)}, got {act!r}")
    return _ACTS[act]


def _columns(x):
    if x.dim() == 0 or x.shape[-1] == 0:
        raise ValueError("expected at least one column")


def _alike(name, t, x):
    if t is not None and (t.shape != x.shape or t.dtype != x.dtype):
        raise ValueError(f"{name} must have the other tensor's shape and type, got {tuple(t.shape)} {t.dtype} for "
                         f"{tuple(x.shape)} {x.dtype}")


def _opt_rows(t):
    return (None, 0) if t is None else _rows(t)


# ---- the norms around a block

def _norm_inputs(x, residual, post_gamma, pre_gamma, gate):
    """x, residual and gate as matrices with leading dimensions (a gate of one row: 0), packed gains."""
    _on_gpu(x, residual, post_gamma, pre_gamma, gate)
    _columns(x)
    _dt(x)
    _alike("residual", residual, x)
    for name, g in (("post_gamma", post_gamma), ("pre_gamma", pre_gamma)):
        if g.shape != x.shape[-1:]:
            raise ValueError(f"{name} must have the shape of x's last dimension, got {tuple(g.shape)} for {tuple(x.shape)}")
    if post_gamma.dtype != pre_gamma.dtype:
        raise ValueError(f"the gains must have one type, got {post_gamma.dtype} and {pre_gamma.dtype}")
    if gate is not None and (gate.dtype != x.dtype or gate.shape not in (x.shape, x.shape[-1:])):
        raise ValueError(f"gate must have x's type, and x's shape or that of its last dimension, got {tuple(gate.shape)} "
                         f"{gate.dtype} for {tuple(x.shape)} {x.dtype}")
    g, ld_g = None, 0
    if gate is not None:
        # one row for all: also where x itself is one row of as many dimensions
        g, ld_g = (gate.contiguous(), 0) if gate.dim() == 1 else _rows(gate)
    return _rows(x), _opt_rows(residual), (g, ld_g), post_gamma.contiguous(), pre_gamma.contiguous()


class _BlockNorms(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, residual, post_gamma, pre_gamma, gate, sigmoid, scale, eps):
        (m, ld), (r, ld_r), (g, ld_g), post, pre = _norm_inputs(x, residual, post_gamma, pre_gamma, gate)
        rows, cols = m.shape
        dt = _dt(m)
        # tensors of their own: y may be changed in place, and freed, while h is kept
        h = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        y = torch.empty_like(h)
        stats = torch.empty((2, rows), dtype=torch.float32, device=x.device)
        nv.nvfp4_block_norms(m, r, g, dt, rows, cols, ld, ld_r, ld_g, sigmoid, post, pre, _dt(post), eps, scale, h, cols,
                             y, cols, None, 0, None, stats[0], stats[1])
        ctx.set_materialize_grads(False)  # an unused h has no gradient to read
        ctx.save_for_backward(m, h, stats, post, pre, g)
        ctx.meta = (ld, ld_g, sigmoid, scale, residual is not None, x.shape, post_gamma.dtype, gate is None or gate.shape)
        return h, y

    @staticmethod
    @once_differentiable
    def backward(ctx, dh, dy):
        m, h, stats, post, pre, g = ctx.saved_tensors
        ld, ld_g, sigmoid, scale, has_residual, shape, gamma_dtype, gate_shape = ctx.meta
        rows, cols = m.shape
        need_x, need_r, need_post, need_pre, need_g = ctx.needs_input_grad[:5]
        need_r = need_r and has_residual
        if dy is None and dh is None or not (need_x or need_r or need_post or need_pre or need_g):
            return (None,) * 8
        dy, ld_dy = _rows(torch.zeros_like(h) if dy is None else dy)
        dh, ld_dh = _opt_rows(dh)

        def out(need):
            return torch.empty(shape, dtype=h.dtype, device=h.device) if need else None

        def sums(need):
            return torch.empty(cols, dtype=torch.float32, device=h.device) if need else None
        shared = g is not None and ld_g == 0
        dx, dr = out(need_x), out(need_r)
        dg = sums(need_g) if shared else out(need_g)
        dpost, dpre = sums(need_post), sums(need_pre)
        ws = None
        if need_post or need_pre or need_g and shared:
            ws = torch.empty(nv.nvfp4_block_norms_backward_workspace_size(rows, cols), dtype=torch.uint8, device=h.device)
        nv.nvfp4_block_norms_backward(dy, dh, h, m, g, _dt(h), rows, cols, ld_dy, ld_dh, cols, ld, ld_g, sigmoid, post, pre,
                                      _dt(post), stats[0], stats[1], scale, dx, cols, dr, cols, dg, cols, dpost, dpre, ws)
        if dg is not None:
            dg = dg.to(h.dtype).view(gate_shape)
        return (dx, dr, None if dpost is None else dpost.to(gamma_dtype), None if dpre is None else dpre.to(gamma_dtype),
                dg, None, None, None)


def block_norms(x, residual, post_gamma, pre_gamma, gate=None, scale: float = 1.0, sigmoid: bool = False,
                eps: float = 1e-5):
    """(h, y): h = residual + scale * g * rms_norm(x) * post_gamma, y = rms_norm(h) * pre_gamma; residual None is
    zero.  gate has x's shape, or its last dimension's (one gate per channel); g is the gate, its logistic function
    where sigmoid is true, 1 without one."""
    return _BlockNorms.apply(x, residual, post_gamma, pre_gamma, gate, int(bool(sigmoid)), float(scale), float(eps))


class BlockNorms(torch.nn.Module):
    """block_norms with its two gains, and a learned gate per channel where layer_scale (its first value) is given."""

    def __init__(self, features: int, scale: float = 1.0, layer_scale: float | None = None, eps: float = 1e-5,
                 device="cuda", dtype=None):
        super().__init__()
        dtype = dtype or torch.bfloat16
        self.post_gamma, self.pre_gamma = (torch.nn.Parameter(torch.ones(features, device=device, dtype=dtype))
                                           for _ in range(2))
        self.gate = None if layer_scale is None else torch.nn.Parameter(
            torch.full((features,), layer_scale, device=device, dtype=dtype))
        self.scale, self.eps = scale, eps

    def forward(self, x, residual=None, gate=None, sigmoid: bool = False):
        """gate: the block's own (x's shape), where there is no layer scale."""
        if gate is not None and self.gate is not None:
            raise ValueError("BlockNorms has a gate per channel: it takes no other")
        if self.gate is not None:
            gate, sigmoid = self.gate.to(x.dtype), False
        return block_norms(x, residual, self.post_gamma, self.pre_gamma, gate, self.scale, sigmoid, self.eps)


# ---- tensors kept in 8 bits

def _kept(rows, cols, device):
    return (torch.empty((rows, cols), dtype=torch.int8, device=device),
            torch.empty((rows, (cols + 31) // 32), dtype=torch.uint8, device=device))


def keep8(x):
    """(codes, scales): x in 8 bits, int8 codes of x's shape and one scale byte per 32 columns; the value of a code is
    code * 2^(byte - 133)."""
    _on_gpu(x)
    _columns(x)
    m, ld = _rows(x)
    rows, cols = m.shape
    codes, scales = _kept(rows, cols, x.device)
    nv.nvfp4_gated_act(nv.NVFP4_ACT_NONE, m, None, _dt(m), rows, cols, ld, 0, None, 0, codes, scales, None, None)
    return codes.view(x.shape), scales.view(*x.shape[:-1], scales.shape[1])


def restore8(codes, scales, dtype=torch.bfloat16):
    """The tensor that keep8's codes and scales stand for."""
    _on_gpu(codes, scales)
    _columns(codes)
    lead, cols = codes.shape[:-1], codes.shape[-1]
    if codes.dtype != torch.int8 or scales.dtype != torch.uint8 or scales.shape != (*lead, (cols + 31) // 32):
        raise ValueError(f"expected int8 codes and a uint8 scale per 32 of their columns, got {tuple(codes.shape)} "
                         f"{codes.dtype} and {tuple(scales.shape)} {scales.dtype}")
    y = torch.empty(codes.shape, dtype=dtype, device=codes.device)
    nv.nvfp4_gated_act_backward(nv.NVFP4_ACT_NONE, codes.contiguous(), scales.contiguous(), None, None, None, _dt(y),
                                y.numel() // cols, cols, 0, None, 0, None, 0, y, cols)
    return y


def _act_forward(gate, up, act, save):
    """y and the kept (codes, scales) of gate and up."""
    _on_gpu(gate, up)
    _columns(gate)
    _alike("up", up, gate)
    g, ld_g = _rows(gate)
    u, ld_u = _opt_rows(up)
    rows, cols = g.shape
    y = torch.empty(gate.shape, dtype=gate.dtype, device=gate.device)
    gc, gs, uc, us = (None,) * 4
    if save:
        gc, gs = _kept(rows, cols, gate.device)
        if up is not None:
            uc, us = _kept(rows, cols, gate.device)
    nv.nvfp4_gated_act(act, g, u, _dt(g), rows, cols, ld_g, ld_u, y, cols, gc, gs, uc, us)
    return y, (gc, gs, uc, us)


def _act_backward(act, kept, dy, shape, need_gate, need_up, need_y):
    """dgate, dup, y of the kept inputs, each where it is needed, of dy's type."""
    gc, gs, uc, us = kept
    rows, cols = gc.shape
    need_up = need_up and uc is not None
    d, ld = _rows(dy) if need_gate or need_up else (None, 0)
    dg, du, y = (torch.empty(shape, dtype=dy.dtype, device=dy.device) if need else None
                 for need in (need_gate, need_up, need_y))
    nv.nvfp4_gated_act_backward(act, gc, gs, uc, us, d, _dt(dy), rows, cols, ld, dg, cols, du, cols, y, cols)
    return dg, du, y


class _GatedAct(torch.autograd.Function):
    @staticmethod
    def forward(ctx, gate, up, act, grad):
        y, kept = _act_forward(gate, up, act, grad and any(ctx.needs_input_grad))
        ctx.save_for_backward(*kept)
        ctx.act = act
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        need_gate, need_up = ctx.needs_input_grad[:2]
        if not (need_gate or need_up):
            return (None,) * 4
        dg, du, _ = _act_backward(ctx.act, ctx.saved_tensors, dy, dy.shape, need_gate, need_up, False)
        return dg, du, None, None


def gated_act(gate, up=None, act: str = "silu"):
    """act(gate) * up (up None: act(gate)); act one of none, silu, gelu (the tanh form), relu2.  What the backward
    pass needs of gate and up is kept in 8 bits: the gradients are those at the kept values."""
    return _GatedAct.apply(gate, up, _act_code(act), torch.is_grad_enabled())


class _GatedActLinear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, gate, up, w, act, grad):
        _on_gpu(w)
        if w.dim() != 2 or w.shape[0] == 0 or w.dtype != gate.dtype or gate.shape[-1:] != w.shape[1:]:
            raise ValueError(f"expected a weight [out, {gate.shape[-1] if gate.dim() else 0}] of the gate's type, got "
                             f"{tuple(w.shape)} {w.dtype}")
        a, kept = _act_forward(gate, up, act, grad and any(ctx.needs_input_grad))
        ctx.save_for_backward(w, *kept)
        ctx.act = act
        return torch.nn.functional.linear(a, w)

    @staticmethod
    @once_differentiable
    def backward(ctx, dz):
        w, *kept = ctx.saved_tensors
        need_gate, need_up, need_w = ctx.needs_input_grad[:3]
        if not (need_gate or need_up or need_w):
            return (None,) * 5
        shape = (*dz.shape[:-1], w.shape[1])
        dz = dz.reshape(-1, w.shape[0])
        # under autocast dz has the product's type, which its other factors then take as well
        da = (dz @ w.to(dz.dtype)).to(w.dtype) if need_gate or need_up else w
        dg, du, a = _act_backward(ctx.act, kept, da, shape, need_gate, need_up, need_w)
        dw = (dz.t() @ a.view(-1, w.shape[1]).to(dz.dtype)).to(w.dtype) if need_w else None
        return dg, du, dw, None, None


def gated_act_linear(gate, up, weight, act: str = "silu"):
    """gated_act(gate, up, act) @ weight^T for a layer that stays in BF16 (or FP32; torch's product, under autocast in its
    type): the activation, which the weight's gradient takes, is not kept but formed again from gate's and up's 8 bits."""
    return _GatedActLinear.apply(gate, up, weight, _act_code(act), torch.is_grad_enabled())


# ---- the product of 8-bit integers

def _pad16(n: int) -> int:
    return (n + 15) // 16 * 16


def _no_grad(*tensors):
    if torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in tensors):
        raise RuntimeError("the 8-bit product has no gradient: call it under torch.no_grad(), or detach its inputs")


def _code_rows(rows, K, device):
    """Rows of K codes, each starting on a line of 128 bytes: the product reads those whole (1 x 20480 x 5136 19.0 us,
    25.0 with rows next to each other; 8192 x 5120 x 5136 232 and 265)."""
    return torch.empty((rows, (K + 127) // 128 * 128), dtype=torch.int8, device=device)[:, :K]


def _code_buffers(rows, cols, device):
    return _code_rows(rows, _pad16(cols), device), torch.empty(rows, dtype=torch.float32, device=device)


def int8_quantize(x):
    """(codes, scales) of x's rows: int8 codes [rows, columns up to a multiple of 16] (zeros past the last column; rows
    start on 128-byte lines), one FP32 scale per row."""
    _no_grad(x)
    _on_gpu(x)
    _columns(x)
    m, ld = _rows(x)
    rows, cols = m.shape
    codes, scales = _code_buffers(rows, cols, x.device)
    nv.nvfp4_int8_quantize(m, _dt(m), rows, cols, ld, codes, codes.stride(0), scales)
    return codes, scales


def int8_quantize_gated(gate, up=None, act: str = "silu"):
    """int8_quantize of gated_act(gate, up, act), in one pass and from its unrounded values."""
    act = _act_code(act)
    _no_grad(gate, up)
    _on_gpu(gate, up)
    _columns(gate)
    _alike("up", up, gate)
    g, ld_g = _rows(gate)
    u, ld_u = _opt_rows(up)
    rows, cols = g.shape
    codes, scales = _code_buffers(rows, cols, gate.device)
    nv.nvfp4_int8_quantize_gated(act, g, u, _dt(g), rows, cols, ld_g, ld_u, codes, codes.stride(0), scales)
    return codes, scales


def block_norms_int8(x, residual, post_gamma, pre_gamma, gate=None, scale: float = 1.0, sigmoid: bool = False,
                     eps: float = 1e-5):
    """(h, codes, scales): block_norms with y as int8_quantize would give it (from its unrounded values)."""
    _no_grad(x, residual, post_gamma, pre_gamma, gate)
    (m, ld), (r, ld_r), (g, ld_g), post, pre = _norm_inputs(x, residual, post_gamma, pre_gamma, gate)
    rows, cols = m.shape
    h = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    codes, scales = _code_buffers(rows, cols, x.device)
    nv.nvfp4_block_norms(m, r, g, _dt(m), rows, cols, ld, ld_r, ld_g, int(bool(sigmoid)), post, pre, _dt(post), float(eps),
                         float(scale), h, cols, None, 0, codes, codes.stride(0), scales, None, None)
    return h, codes, scales


def int8_matmul(codes, scales, w_codes, w_scales, dtype=torch.bfloat16):
    """codes w_codes^T times their scales: [rows, out] of the given type."""
    _no_grad(scales, w_scales)
    _on_gpu(codes, scales, w_codes, w_scales)
    if codes.dim() != 2 or w_codes.dim() != 2 or codes.shape[1] != w_codes.shape[1] or codes.shape[1] % 16 != 0 \
            or codes.shape[1] == 0:
        raise ValueError(f"expected codes [rows, K] and [out, K] with K a multiple of 16, got {tuple(codes.shape)} and "
                         f"{tuple(w_codes.shape)}")
    for c, s in ((codes, scales), (w_codes, w_scales)):
        if c.dtype != torch.int8 or s.dtype != torch.float32 or s.shape != c.shape[:1]:
            raise ValueError(f"expected int8 codes and a float32 scale per row, got {tuple(c.shape)} {c.dtype} and "
                             f"{tuple(s.shape)} {s.dtype}")
    M, K = codes.shape
    N = w_codes.shape[0]

    def operand(t):  # as it lies where its rows are 16-byte pieces
        ok = (t.stride(1) == 1 and t.stride(0) >= K and t.stride(0) % 16 == 0 and t.stride(0) < 2 ** 23
              and t.data_ptr() % 16 == 0)
        return t if ok else t.clone(memory_format=torch.contiguous_format)
    a, b = operand(codes), operand(w_codes)
    y = torch.empty((M, N), dtype=dtype, device=codes.device)
    if N == 0:
        return y
    ws = torch.empty(nv.nvfp4_int8_gemm_workspace_size(M, N, K), dtype=torch.uint8, device=codes.device)
    nv.nvfp4_int8_gemm(M, N, K, a, max(a.stride(0), K), scales.contiguous(), b, max(b.stride(0), K), w_scales.contiguous(),
                       y, _dt(y), N, ws)
    return y


class Int8Linear(torch.nn.Module):
    """Bias-free linear layer for inference: its weight in 8 bits with a scale per output channel (buffers, quantized
    once), its input quantized per token on each call."""

    def __init__(self, weight):
        super().__init__()
        if weight.dim() != 2:
            raise ValueError(f"expected a weight [out, in], got {tuple(weight.shape)}")
        self.out_features, self.in_features = weight.shape
        codes, scales = int8_quantize(weight.detach())
        self.register_buffer("codes", codes)
        self.register_buffer("scales", scales)

    @classmethod
    def from_linear(cls, layer):
        """From a layer with a weight [out, in] and no bias (NVFP4Linear, torch.nn.Linear)."""
        if getattr(layer, "bias", None) is not None:
            raise ValueError("Int8Linear has no bias")
        return cls(layer.weight)

    def _apply(self, fn, recurse=True):
        scales = self.scales
        super()._apply(fn, recurse)
        if self.scales.dtype != torch.float32:  # a change of the model's type leaves the scales in FP32
            self.scales = scales.to(self.scales.device)
        if self.codes.stride(0) % 128 != 0:  # a copy has packed the rows
            self.codes = _code_rows(*self.codes.shape, self.codes.device).copy_(self.codes)
        return self

    def _inputs(self, x):
        if x.dim() == 0 or x.shape[-1] != self.in_features:
            raise ValueError(f"expected {self.in_features} columns, got {tuple(x.shape)}")

    def _product(self, codes, scales, x):
        return int8_matmul(codes, scales, self.codes, self.scales, x.dtype).view(*x.shape[:-1], self.out_features)

    def forward(self, x):
        self._inputs(x)
        return self._product(*int8_quantize(x), x)

    def gated(self, gate, up=None, act: str = "silu"):
        """The layer of gated_act(gate, up, act)."""
        self._inputs(gate)
        return self._product(*int8_quantize_gated(gate, up, act), gate)

    def normed(self, x, residual, post_gamma, pre_gamma, gate=None, scale: float = 1.0, sigmoid: bool = False,
               eps: float = 1e-5):
        """(h, the layer of y) of block_norms."""
        self._inputs(x)
        h, codes, scales = block_norms_int8(x, residual, post_gamma, pre_gamma, gate, scale, sigmoid, eps)
        return h, self._product(codes, scales, x)
