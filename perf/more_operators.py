"""Cases that time the operators of a residual block in eight bits: the product of 8-bit integers
with a scale per token and per output channel (with the quantization of its input, from a tensor,
a gated activation or the norms around a block), the two norms around a block with its gate and
residual scale and their backward pass, and the gated activation whose inputs are kept in 8 bits
for its backward pass.

`run` computes each case in plain torch operations where `own` is false and through the
library's entry points where it is true; `exact` computes it from the definition in 64 bits.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-5
BLOCK = 32  # elements per scale of a kept activation
ACTS = ("none", "silu", "gelu", "relu2")


def listed():
    return [
        # one token being served: norms around a block, 8-bit input, the next block's up-projection
        dict(name="int8_token", op="int8", src="norms", M=1, N=20480, K=5120, dt="bf16", act="none", pad=0),
        # a batch of sequences, one new token each: gated activation and down-projection
        dict(name="int8_batch", op="int8", src="gated", M=48, N=5120, K=20480, dt="bf16", act="silu", pad=0),
        # a short prompt through a pruned layer of odd sizes, FP32 in and out
        dict(name="int8_odd", op="int8", src="x", M=257, N=4999, K=2047, dt="f32", act="none", pad=3),
        # a long prompt: up-projection of a chunk of tokens
        dict(name="int8_prompt", op="int8", src="x", M=8192, N=20480, K=5120, dt="bf16", act="none", pad=0),
        # the norms of a few tokens being served: latency of one call
        dict(name="norms_short", op="norms", rows=16, cols=5120, pad=0, dt="bf16", gate="none"),
        # forward of a training step: a gate per token and channel, kept statistics
        dict(name="norms_train", op="norms", rows=8192, cols=5120, pad=0, dt="bf16", gate="token"),
        # its backward pass: gradients of the block's output, the residual, the gate and both gains
        dict(name="norms_back", op="norms_back", rows=8192, cols=5120, pad=0, dt="bf16", gate="token"),
        # FP32 at an odd width, one gate per channel (a learned layer scale)
        dict(name="norms_back_f32_odd", op="norms_back", rows=1023, cols=8191, pad=0, dt="f32", gate="channel"),
        # the activation of a short micro-batch without a second branch: latency of one call
        dict(name="act_short", op="act", rows=64, cols=5120, pad=0, dt="bf16", act="relu2", gated=False),
        # the widest activation of a training step, both branches kept in 8 bits
        dict(name="act_train", op="act", rows=8192, cols=20480, pad=0, dt="bf16", act="silu", gated=True),
        # its backward pass, the activation itself formed again for the next weight gradient
        dict(name="act_back", op="act_back", rows=8192, cols=20480, pad=0, dt="bf16", act="silu", gated=True,
             again=True),
        # FP32 at an odd width, gradients written into slices of a wider buffer (a fused projection's)
        dict(name="act_back_f32_slice", op="act_back", rows=1025, cols=5119, pad=5121, dt="f32", act="gelu",
             gated=True, again=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["int8", "int8", "norms", "norms_back", "act", "act_back"])
    dt = rng.choice(["bf16", "bf16", "f32"])
    if op == "int8":
        src = rng.choice(["x", "gated", "norms"])
        M, N = _log(rng, 1, 8192), _log(rng, 64, 20480)
        K = _log(rng, 128, 8192 if src == "norms" else 20480)
        if rng.random() < 0.6:  # sizes that a model has, beside odd ones
            N, K = max(64, N // 64 * 64), max(128, K // 128 * 128)
        K = min(K, 8192 * 20480 * 5120 // (M * N))
        return dict(op=op, src=src, M=M, N=N, K=K, dt=dt, act=rng.choice(ACTS[1:]) if src == "gated" else "none",
                    pad=rng.choice([0, 0, 1, 8]))
    norms = op.startswith("norms")
    rows, cols = _log(rng, 1, 32768), _log(rng, 128, 8192 if norms else 20480)
    rows = min(rows, 8192 * (5120 if norms else 20480) // cols)
    if rng.random() < 0.5:
        cols = max(128, cols // 64 * 64)
    case = dict(op=op, rows=rows, cols=cols, pad=rng.choice([0, 0, 1, 8, 64]), dt=dt)
    if norms:
        case["gate"] = rng.choice(["none", "channel", "token"])
        return case
    case.update(act=rng.choice(ACTS[1:]), gated=rng.random() < 0.7)
    if op == "act_back":
        case["again"] = rng.random() < 0.5
    return case


# ---- inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(g, rows, cols, dt, pad=0, std=1.0):
    """N(0, std^2), one channel in a thousand ten times as large, as hidden states have them;
    `pad` columns of a wider buffer follow each row."""
    buf = torch.empty((rows, cols + pad), dtype=dt, device="cuda")
    v = torch.randn((rows, cols), generator=g, device="cuda")
    gain = torch.full((cols,), std, device="cuda")
    gain[torch.randint(cols, (cols // 1000 + 1,), generator=g, device="cuda")] *= 10.0
    x = buf[:, :cols]
    x.copy_(v.mul_(gain))
    return x


def _wider(rows, cols, dt, pad):
    """An output of rows x cols in a buffer whose rows are `pad` columns longer."""
    return torch.empty((rows, cols + pad), dtype=dt, device="cuda")[:, :cols]


def _gain(g, cols, dt):
    return (1.0 + 0.2 * torch.randn(cols, generator=g, device="cuda")).to(dt)


def _norm_inputs(s, g, rows, cols, dt, pad, gate):
    s["x"] = _normal(g, rows, cols, dt, pad)
    s["residual"] = _normal(g, rows, cols, dt, pad, 3.0)
    s["post"], s["pre"] = _gain(g, cols, dt), _gain(g, cols, dt)
    s["scale"] = 0.75
    s["gate_in"] = None
    if gate == "token":
        s["gate_in"] = _normal(g, rows, cols, dt, pad)
    elif gate == "channel":
        s["gate_in"] = (0.5 + 0.2 * torch.randn(cols, generator=g, device="cuda")).to(dt)


def _out(case):
    """Type of a product: BF16 behind a gated activation or the norms, whose FP32 values are
    rounded to integers, so that one in some 10^5 falls to either side of a border."""
    return DT[case["dt"]] if case["src"] == "x" else torch.bfloat16


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case)
    dt, pad = DT[case["dt"]], case["pad"]
    if case["op"] == "int8":
        M, N, K = case["M"], case["N"], case["K"]
        Kp = (K + 15) // 16 * 16  # rows of codes are whole 16-byte pieces, zeros at their end
        w = torch.randn((N, K), generator=g, device="cuda")
        w.mul_(0.02 * (0.5 + torch.rand((N, 1), generator=g, device="cuda")))
        top = w.abs().amax(1, keepdim=True)
        s["w"] = torch.zeros((N, Kp), dtype=torch.int8, device="cuda")
        s["w"][:, :K] = torch.round(w.mul_(127.0 / top)).to(torch.int8)
        s["w_scales"] = top[:, 0] / 127.0
        if case["src"] == "norms":
            _norm_inputs(s, g, M, K, dt, pad, "none")
            s["h"] = torch.empty((M, K), dtype=dt, device="cuda")
        else:
            s["x"] = _normal(g, M, K, dt, pad)
            if case["src"] == "gated":
                s["up"] = _normal(g, M, K, dt, pad)
        s["codes"] = torch.empty((M, Kp), dtype=torch.int8, device="cuda")
        s["scales"] = torch.empty(M, device="cuda")
        s["y"] = torch.empty((M, N), dtype=_out(case), device="cuda")
        return s
    rows, cols = case["rows"], case["cols"]
    if case["op"] in ("norms", "norms_back"):
        _norm_inputs(s, g, rows, cols, dt, pad, case["gate"])
        s["post_rstd"], s["pre_rstd"] = (torch.empty(rows, device="cuda") for _ in range(2))
        if case["op"] == "norms":
            s["h"], s["y"] = (torch.empty((rows, cols), dtype=dt, device="cuda") for _ in range(2))
            return s
        # the saved sum and statistics; gradients of a training step's magnitude
        h, _, s["post_rstd"], s["pre_rstd"] = _norms(s)
        s["h"] = h.to(dt)
        del s["residual"]
        s["dy"], s["dh"] = (_normal(g, rows, cols, dt, pad, 1e-3) for _ in range(2))
        s["dx"], s["dresidual"] = (torch.empty((rows, cols), dtype=dt, device="cuda") for _ in range(2))
        s["dpost"], s["dpre"] = (torch.empty(cols, device="cuda") for _ in range(2))
        s["dgate"] = None
        if case["gate"] == "token":
            s["dgate"] = torch.empty((rows, cols), dtype=dt, device="cuda")
        elif case["gate"] == "channel":
            s["dgate"] = torch.empty(cols, device="cuda")
        return s
    inputs = ["gate", "up"] if case["gated"] else ["gate"]
    for name in inputs:
        v = _normal(g, rows, cols, dt, pad if case["op"] == "act" else 0, 1.0)
        if case["op"] == "act":
            s[name] = v
            s[name + "_codes"] = torch.empty((rows, cols), dtype=torch.int8, device="cuda")
            s[name + "_scales"] = torch.empty((rows, -(-cols // BLOCK)), dtype=torch.uint8, device="cuda")
        else:
            s[name + "_codes"], s[name + "_scales"] = _keep(v.float())
            s["d" + name] = _wider(rows, cols, dt, pad)
    s["y"] = torch.empty((rows, cols), dtype=dt, device="cuda") if case.get("again", True) else None
    if case["op"] == "act_back":
        s["dy"] = _normal(g, rows, cols, dt, 0, 1e-3)
    return s


# ---- the plain forms

def _act(name, v):
    """act(v) in FP32."""
    if name == "silu":
        return v / (1.0 + torch.exp(-v))
    if name == "gelu":
        t = 0.7978845608028654 * (v + 0.044715 * v * v * v)
        return v / (1.0 + torch.exp(-2.0 * t))  # (1 + tanh t) / 2 = 1 / (1 + exp(-2 t))
    if name == "relu2":
        return torch.where(v > 0, v * v, torch.zeros_like(v))
    return v


def _slope(name, v):
    """The derivative of act at v in FP32."""
    if name == "silu":
        p = 1.0 / (1.0 + torch.exp(-v))
        return p * (1.0 + v * (1.0 - p))
    if name == "gelu":
        t = 0.7978845608028654 * (v + 0.044715 * v * v * v)
        p = 1.0 / (1.0 + torch.exp(-2.0 * t))
        return p + v * 2.0 * p * (1.0 - p) * 0.7978845608028654 * (1.0 + 3.0 * 0.044715 * v * v)
    if name == "relu2":
        return torch.where(v > 0, 2.0 * v, torch.zeros_like(v))
    return torch.ones_like(v)


def _sigmoid(v):
    return 1.0 / (1.0 + torch.exp(-v))


def _norms(s):
    """(h, y, post_rstd, pre_rstd) in FP32."""
    x = s["x"].float()
    post = 1.0 / torch.sqrt((x * x).mean(1) + EPS)
    o = (x * post[:, None]) * s["post"].float()
    if s["gate_in"] is not None:
        gate = s["gate_in"].float()
        o = o * (_sigmoid(gate) if s["gate"] == "token" else gate)
    h = s["residual"].float() + s["scale"] * o
    pre = 1.0 / torch.sqrt((h * h).mean(1) + EPS)
    return h, (h * pre[:, None]) * s["pre"].float(), post, pre


def _quantized(v):
    """Codes and scale of each row: the scale is its largest magnitude / 127, the code the
    nearest integer to v * (127 / largest).  (Tensor / tensor: a division, where a Python
    number on either side becomes a product with its reciprocal.)"""
    top = v.abs().amax(1)
    most = torch.full_like(top, 127.0)
    live = top >= 2.0 ** -100
    inv = torch.where(live, most / top, torch.zeros_like(top))
    return torch.round(v * inv[:, None]), torch.where(live, top / most, torch.zeros_like(top))


def _keep(v):
    """Codes and scale bytes of blocks of 32 along the rows: value = code * 2^(byte - 133), the
    smallest byte in [0, 254] under which no code of the block exceeds 127."""
    rows, cols = v.shape
    blocks = -(-cols // BLOCK)
    b = torch.nn.functional.pad(v, (0, blocks * BLOCK - cols)).view(rows, blocks, BLOCK)
    m, ex = torch.frexp(b.abs().amax(2))  # m in [0.5, 1): m * 2^ex <= 127 * 2^e
    e = torch.where(m <= 127.0 / 128.0, ex - 7, ex - 6)
    e = torch.where(m == 0, torch.full_like(e, -133), e.clamp(-133, 121))
    q = torch.round(b.double() * torch.exp2(-e.double())[:, :, None])  # exact: up to 2^133
    codes = q.to(torch.int8).view(rows, blocks * BLOCK)[:, :cols].contiguous()
    return codes, (e + 133).to(torch.uint8)


def _kept(codes, scales):
    """The values that codes and scale bytes stand for, FP32."""
    step = torch.exp2(scales.double() - 133.0).float()
    return codes.float() * step.repeat_interleave(BLOCK, 1)[:, :codes.shape[1]]


def _plain(s):
    dt = DT[s["dt"]]
    if s["op"] == "int8":
        out = {}
        if s["src"] == "norms":
            h, v, _, _ = _norms(s)
            out["h"] = h.to(dt)
        else:
            v = _act(s["act"], s["x"].float())
            if s["src"] == "gated":
                v = v * s["up"].float()
        q, scale = _quantized(v)
        # sums of whole numbers up to 127^2 K: exact in 64 bits
        z = (q.double() @ s["w"][:, :s["K"]].double().t()).float()
        if s["src"] == "x":
            short = s["codes"].shape[1] - s["K"]
            out["codes"], out["scales"] = torch.nn.functional.pad(q, (0, short)).to(torch.int8), scale
        out["y"] = ((z * s["w_scales"]) * scale[:, None]).to(_out(s))
        return out
    if s["op"] == "norms":
        h, y, post, pre = _norms(s)
        return dict(h=h.to(dt), y=y.to(dt), post_rstd=post, pre_rstd=pre)
    if s["op"] == "norms_back":
        h, x, dy = s["h"].float(), s["x"].float(), s["dy"].float()
        post, pre = s["post_rstd"][:, None], s["pre_rstd"][:, None]
        n = h * pre
        a = dy * s["pre"].float()
        dr = s["dh"].float() + pre * (a - n * (a * n).mean(1, keepdim=True))
        out = dict(dresidual=dr.to(dt), dpre=(dy * n).sum(0))
        n = x * post
        do = s["scale"] * dr
        if s["gate_in"] is not None:
            raw = s["gate_in"].float()
            gate = _sigmoid(raw) if s["gate"] == "token" else raw
            d = do * n * s["post"].float()
            out["dgate"] = (d * (gate * (1.0 - gate))).to(dt) if s["gate"] == "token" else d.sum(0)
            do = do * gate
        out["dpost"] = (do * n).sum(0)
        b = do * s["post"].float()
        out["dx"] = (post * (b - n * (b * n).mean(1, keepdim=True))).to(dt)
        return out
    if s["op"] == "act":
        gate = s["gate"].float()
        y = _act(s["act"], gate)
        out = {}
        out["gate_codes"], out["gate_scales"] = _keep(gate)
        if s["gated"]:
            up = s["up"].float()
            y = y * up
            out["up_codes"], out["up_scales"] = _keep(up)
        out["y"] = y.to(dt)
        return out
    dy, gate = s["dy"].float(), _kept(s["gate_codes"], s["gate_scales"])
    a, slope = _act(s["act"], gate), _slope(s["act"], gate)
    out = {}
    if s["gated"]:
        up = _kept(s["up_codes"], s["up_scales"])
        out["dup"] = (dy * a).to(dt)
        a, dy = a * up, dy * up
    out["dgate"] = (dy * slope).to(dt)
    if s["again"]:
        out["y"] = a.to(dt)
    return out


# ---- the library's entry points

def _library(s):
    import bit_microscaled_quantized_amd as nv
    code = nv.NVFP4_F32 if s["dt"] == "f32" else nv.NVFP4_BF16
    acts = dict(none=nv.NVFP4_ACT_NONE, silu=nv.NVFP4_ACT_SILU, gelu=nv.NVFP4_ACT_GELU, relu2=nv.NVFP4_ACT_RELU2)

    def ld(t):
        return 0 if t is None else t.stride(0)

    if s["op"] == "int8":
        M, N, K, x, c, sc, y = s["M"], s["N"], s["K"], s["x"], s["codes"], s["scales"], s["y"]
        Kp = c.shape[1]
        if s["src"] == "norms":
            r, h = s["residual"], s["h"]
            nv.nvfp4_block_norms(x, r, None, code, M, K, ld(x), ld(r), 0, nv.NVFP4_GATE_LINEAR, s["post"], s["pre"],
                                 code, EPS, s["scale"], h, ld(h), None, 0, c, Kp, sc, None, None)
        elif s["src"] == "gated":
            nv.nvfp4_int8_quantize_gated(acts[s["act"]], x, s["up"], code, M, K, ld(x), ld(s["up"]), c, Kp, sc)
        else:
            nv.nvfp4_int8_quantize(x, code, M, K, ld(x), c, Kp, sc)
        ws = torch.empty(nv.nvfp4_int8_gemm_workspace_size(M, N, Kp), dtype=torch.uint8, device="cuda")
        out = nv.NVFP4_F32 if y.dtype == torch.float32 else nv.NVFP4_BF16
        nv.nvfp4_int8_gemm(M, N, Kp, c, Kp, sc, s["w"], Kp, s["w_scales"], y, out, N, ws)
        return dict(dict(h=s["h"]) if s["src"] == "norms" else dict(codes=c, scales=sc) if s["src"] == "x" else {}, y=y)
    rows, cols = s["rows"], s["cols"]
    if s["op"].startswith("norms"):
        x, gate = s["x"], s["gate_in"]
        ld_gate = ld(gate) if s["gate"] == "token" else 0  # 0: one row of gates for all
        kind = nv.NVFP4_GATE_SIGMOID if s["gate"] == "token" else nv.NVFP4_GATE_LINEAR
        if s["op"] == "norms":
            r, h, y = s["residual"], s["h"], s["y"]
            nv.nvfp4_block_norms(x, r, gate, code, rows, cols, ld(x), ld(r), ld_gate, kind, s["post"], s["pre"], code,
                                 EPS, s["scale"], h, ld(h), y, ld(y), None, 0, None, s["post_rstd"], s["pre_rstd"])
            return dict(h=h, y=y, post_rstd=s["post_rstd"], pre_rstd=s["pre_rstd"])
        dy, dh, h, dx, dr, dgate = s["dy"], s["dh"], s["h"], s["dx"], s["dresidual"], s["dgate"]
        ws = torch.empty(nv.nvfp4_block_norms_backward_workspace_size(rows, cols), dtype=torch.uint8, device="cuda")
        nv.nvfp4_block_norms_backward(dy, dh, h, x, gate, code, rows, cols, ld(dy), ld(dh), ld(h), ld(x), ld_gate,
                                      kind, s["post"], s["pre"], code, s["post_rstd"], s["pre_rstd"], s["scale"], dx,
                                      ld(dx), dr, ld(dr), dgate, ld(dgate) if s["gate"] == "token" else 0, s["dpost"],
                                      s["dpre"], ws)
        out = dict(dresidual=dr, dpre=s["dpre"], dpost=s["dpost"], dx=dx)
        return out if dgate is None else dict(out, dgate=dgate)
    act, y = acts[s["act"]], s["y"]
    gc, gs, uc, us = (s.get(n) for n in ("gate_codes", "gate_scales", "up_codes", "up_scales"))
    if s["op"] == "act":
        gate, up = s["gate"], s.get("up")
        nv.nvfp4_gated_act(act, gate, up, code, rows, cols, ld(gate), ld(up), y, ld(y), gc, gs, uc, us)
        out = dict(gate_codes=gc, gate_scales=gs, y=y)
        return dict(out, up_codes=uc, up_scales=us) if s["gated"] else out
    dy, dg, du = s["dy"], s["dgate"], s.get("dup")
    nv.nvfp4_gated_act_backward(act, gc, gs, uc, us, dy, code, rows, cols, ld(dy), dg, ld(dg), du, ld(du), y, ld(y))
    out = dict(dgate=dg)
    if s["gated"]:
        out["dup"] = du
    return dict(out, y=y) if s["again"] else out


def run(state):
    return _library(state) if own else _plain(state)


def work(case):
    size = 4 if case["dt"] == "f32" else 2
    if case["op"] == "int8":
        M, N, K = case["M"], case["N"], case["K"]
        out = 4 if _out(case) == torch.float32 else 2
        read = {"x": 1, "gated": 2, "norms": 3}[case["src"]] * M * K * size  # norms: x, residual and h
        return dict(bytes=read + N * K + 4 * N + M * N * out, flops=2 * M * N * K)
    rows, cols = case["rows"], case["cols"]
    n = rows * cols
    if case["op"] in ("norms", "norms_back"):
        back = case["op"] == "norms_back"
        token, channel = case["gate"] == "token", case["gate"] == "channel"
        tensors = (6 if back else 4) + ((2 if back else 1) if token else 0)
        vectors = cols * (2 * size + (8 if back else 0) + (size + (4 if back else 0) if channel else 0))
        return dict(bytes=tensors * n * size + vectors + 8 * rows, flops=(25 if back else 12) * n)
    branches = 2 if case["gated"] else 1
    kept = branches * (n + rows * -(-cols // BLOCK))
    tensors = branches + (1 if case["op"] == "act" or case["again"] else 0) + (1 if case["op"] == "act_back" else 0)
    return dict(bytes=kept + tensors * n * size, flops=12 * branches * n)


# ---- the definitions in 64 bits, written apart from the plain forms

def _act64(name, v):
    """(act(v), its derivative)."""
    if name == "silu":
        p = torch.sigmoid(v)
        return v * p, p + v * p * torch.sigmoid(-v)
    if name == "gelu":
        c = math.sqrt(2.0 / math.pi)
        t = torch.tanh(c * (v + 0.044715 * v.pow(3)))
        return 0.5 * v * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * v * (1.0 - t * t) * c * (1.0 + 0.134145 * v.pow(2))
    if name == "relu2":
        p = v.clamp(min=0.0)
        return p.pow(2), 2.0 * p
    return v, torch.ones_like(v)


def _norm64(x, gamma):
    rstd = (torch.linalg.vecdot(x, x) / x.shape[1] + EPS).pow(-0.5)
    return torch.einsum("rc,r,c->rc", x, rstd, gamma), rstd


def _norms64(s):
    o, post = _norm64(s["x"].double(), s["post"].double())
    if s.get("gate") == "token":
        o = o * torch.sigmoid(s["gate_in"].double())
    elif s.get("gate") == "channel":
        o = o * s["gate_in"].double()
    h = torch.add(s["residual"].double(), o, alpha=s["scale"])
    y, pre = _norm64(h, s["pre"].double())
    return h, y, post, pre


def _norm_grad64(d, v, gamma, rstd):
    """(gradient of v, of gamma) of the norm of v for the gradient d."""
    a = d * gamma
    c = torch.linalg.vecdot(a, v) * rstd.pow(3) / v.shape[1]
    return (torch.einsum("rc,r->rc", a, rstd) - torch.einsum("rc,r->rc", v, c), torch.einsum("rc,rc,r->c", d, v, rstd))


def _kept64(v):
    """(codes, bytes) of the kept form, from the exponents' definition."""
    rows, cols = v.shape
    blocks = torch.cat((v, v.new_zeros(rows, -cols % BLOCK)), 1).unflatten(1, (-1, BLOCK))
    top = blocks.abs().max(2).values
    e = torch.ceil(torch.log2(top / 127.0))
    e = torch.where(top > torch.pow(2.0, e) * 127.0, e + 1, e)
    e = torch.where(top <= torch.pow(2.0, e - 1) * 127.0, e - 1, e).clamp(-133, 121)
    codes = torch.round(blocks / torch.pow(2.0, e)[..., None])
    return codes.flatten(1)[:, :cols], e + 133


def _held64(codes, scales):
    at = torch.arange(codes.shape[1], device="cuda") // BLOCK
    return codes.double() * torch.pow(2.0, scales.double() - 133.0)[:, at]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "int8":
        out = {}
        if case["src"] == "norms":
            out["h"], v, _, _ = _norms64(s)
        else:
            v, _ = _act64(case["act"], s["x"].double())
            if case["src"] == "gated":
                v = v * s["up"].double()
        # a code is defined by two FP32 roundings, of 127 / largest and of its product with the
        # value (which has 48 bits and is exact here before the second)
        top = v.abs().max(1, keepdim=True).values
        step = top / 127.0
        q = torch.round((v * (127.0 / top).float().double()).float().double())
        z = torch.matmul(q, s["w"][:, :case["K"]].double().transpose(0, 1))
        if case["src"] == "x":
            out["codes"] = torch.cat((q, q.new_zeros(case["M"], -case["K"] % 16)), 1).to(torch.int8)
            out["scales"] = step[:, 0]
        out["y"] = z * step * s["w_scales"].double()
        return out
    if case["op"] == "norms":
        h, y, post, pre = _norms64(s)
        return dict(h=h, y=y, post_rstd=post, pre_rstd=pre)
    if case["op"] == "norms_back":
        h, x = s["h"].double(), s["x"].double()
        post, pre = s["post_rstd"].double(), s["pre_rstd"].double()
        gh, dpre = _norm_grad64(s["dy"].double(), h, s["pre"].double(), pre)
        gh = gh + s["dh"].double()
        out = dict(dresidual=gh, dpre=dpre)
        d = gh * s["scale"]
        if case["gate"] != "none":
            raw = s["gate_in"].double()
            o = torch.einsum("rc,r,c->rc", x, post, s["post"].double())
            if case["gate"] == "token":
                out["dgate"] = d * o * torch.sigmoid(raw) * torch.sigmoid(-raw)
                d = d * torch.sigmoid(raw)
            else:
                out["dgate"] = (d * o).sum(0)
                d = d * raw
        out["dx"], out["dpost"] = _norm_grad64(d, x, s["post"].double(), post)
        return out
    if case["op"] == "act":
        y, _ = _act64(case["act"], s["gate"].double())
        out = {}
        out["gate_codes"], out["gate_scales"] = _kept64(s["gate"].double())
        if case["gated"]:
            y = y * s["up"].double()
            out["up_codes"], out["up_scales"] = _kept64(s["up"].double())
        out["y"] = y
        return out
    y, slope = _act64(case["act"], _held64(s["gate_codes"], s["gate_scales"]))
    d, out = s["dy"].double(), {}
    if case["gated"]:
        up = _held64(s["up_codes"], s["up_scales"])
        out["dup"] = d * y
        y, d = y * up, d * up
    out["dgate"] = d * slope
    if case["again"]:
        out["y"] = y
    return out
