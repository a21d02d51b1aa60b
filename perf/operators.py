"""Cases that time the operators between the quantized layers of a training step, and its loss:
counter-based dropout, the residual + RMS norm (BF16 / FP32 output or E4M3 with block scales,
and its backward pass), and the linear softmax cross entropy over a vocabulary with its gradient.

`run` computes each case in plain torch operations where `own` is false and through the
library's entry points where it is true; `exact` computes it from the definition in 64 bits.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-5
U32 = 0xFFFFFFFF


def listed():
    return [
        # dropout on the embedding of a short micro-batch: latency of one call
        dict(name="dropout_short", op="dropout", rows=64, cols=5120, pad=0, dt="bf16", p=0.1),
        # dropout on the widest activation of a training step (the FFN's inner one)
        dict(name="dropout_ffn", op="dropout", rows=8192, cols=20480, pad=0, dt="bf16", p=0.1),
        # odd widths in FP32, a slice of a wider buffer (fused projections split by columns)
        dict(name="dropout_f32_slice", op="dropout", rows=4097, cols=5119, pad=5121, dt="f32", p=0.25),
        # one token being served: residual addition, norm, 8-bit input of the next product
        dict(name="norm_token_mx8", op="norm", rows=1, cols=5120, pad=0, dt="bf16", p=0.0, out="mx8"),
        # forward of a training step: dropout, residual addition and norm of one chunk
        dict(name="norm_train", op="norm", rows=8192, cols=5120, pad=0, dt="bf16", p=0.1, out="y"),
        # a long prompt being served: 8-bit output
        dict(name="norm_prompt_mx8", op="norm", rows=32768, cols=5120, pad=0, dt="bf16", p=0.0, out="mx8"),
        # backward of the training step's norm, with the residual's gradient and the dropout
        dict(name="norm_back", op="norm_back", rows=8192, cols=5120, pad=0, dt="bf16", p=0.1),
        # the same in FP32 at an odd, wide width (rows start at any alignment)
        dict(name="norm_back_f32_odd", op="norm_back", rows=1023, cols=20479, pad=0, dt="f32", p=0.0),
        # the loss of one scored token: the whole head is read for one row
        dict(name="loss_token", op="loss", T=1, V=131072, H=5120, ignore=0.0, train=False),
        # a fine-tuning micro-batch over a ragged vocabulary, prompt tokens ignored
        dict(name="loss_small", op="loss", T=257, V=49999, H=2048, ignore=0.4, train=True),
        # evaluation of one chunk, an odd number of tokens, many of them ignored
        dict(name="loss_eval", op="loss", T=4095, V=99991, H=5120, ignore=0.5, train=False),
        # the head of a training step: one chunk of tokens, loss and both gradients
        dict(name="loss_train", op="loss", T=8192, V=131072, H=5120, ignore=0.0, train=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["dropout", "norm", "norm_back", "loss"])
    if op == "loss":
        H = 8 * _log(rng, 16, 640)
        H += 8 * (H == 3072)
        return dict(op=op, T=_log(rng, 1, 8192), V=_log(rng, 1000, 131072), H=H,
                    ignore=rng.choice([0.0, 0.1, 0.5, 0.9]), train=rng.random() < 0.6)
    rows, cols = _log(rng, 1, 32768), _log(rng, 128, 20480)
    rows = min(rows, 8192 * 20480 // cols)
    if rng.random() < 0.5:  # widths that a model has, beside odd ones
        cols = max(128, cols // 64 * 64)
    cols += cols == 3072
    rows += rows == 3072
    case = dict(op=op, rows=rows, cols=cols, pad=rng.choice([0, 0, 1, 8, 64]),
                dt=rng.choice(["bf16", "bf16", "f32"]), p=rng.choice([0.0, 0.05, 0.1, 0.5]))
    if op == "dropout" and case["p"] == 0.0:
        case["p"] = 0.2
    if op == "norm":
        case["out"] = rng.choice(["y", "mx8"])
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


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case)
    s["seed"] = (seed * 0x9E3779B97F4A7C15 + 12345) & 0xFFFFFFFFFFFFFFFF
    if case["op"] == "loss":
        T, V, H = case["T"], case["V"], case["H"]
        s["w"] = torch.empty((V, H), dtype=torch.bfloat16, device="cuda").normal_(0.0, 0.02, generator=g)
        # frequent and rare tokens; hidden states that lean towards their label by various amounts
        y = (torch.rand(T, generator=g, device="cuda") ** 3 * V).long().clamp_(max=V - 1)
        lean = torch.rand(T, generator=g, device="cuda") * 8.0 / (0.02 * math.sqrt(H))
        x = torch.randn((T, H), generator=g, device="cuda") + lean[:, None] * s["w"][y].float()
        s["x"] = x.to(torch.bfloat16)
        out = torch.rand(T, generator=g, device="cuda") < case["ignore"]
        s["labels"] = torch.where(out, torch.full_like(y, -100), y)
        valid = (~out).float()
        s["dloss"] = valid / valid.sum().clamp(min=1.0)
        s["loss"] = torch.empty(T, device="cuda")
        s["lse"] = torch.empty(T, device="cuda")
        if case["train"]:
            s["dx"] = torch.empty_like(s["x"])
            s["dw"] = torch.empty_like(s["w"])
        return s
    rows, cols, dt, pad = case["rows"], case["cols"], DT[case["dt"]], case["pad"]
    s["x"] = _normal(g, rows, cols, dt, pad)
    if case["op"] == "dropout":
        s["y"] = torch.empty((rows, cols), dtype=dt, device="cuda")
        return s
    s["gamma"] = (1.0 + 0.2 * torch.randn(cols, generator=g, device="cuda")).to(dt)
    if case["op"] == "norm":
        s["residual"] = _normal(g, rows, cols, dt, pad, 3.0)
        s["h"] = torch.empty((rows, cols), dtype=dt, device="cuda")
        s["rstd"] = torch.empty(rows, device="cuda")
        if case["out"] == "mx8":
            s["codes"] = torch.empty((rows, cols), dtype=torch.float8_e4m3fn, device="cuda")
            s["scales"] = torch.empty((rows, (cols + 31) // 32), dtype=torch.float8_e8m0fnu, device="cuda")
        else:
            s["y"] = torch.empty((rows, cols), dtype=dt, device="cuda")
        return s
    # norm_back: x is the saved sum h; the gradients have a training step's magnitude
    s["h"] = s.pop("x")
    s["rstd"] = (s["h"].float().square().mean(1) + EPS).rsqrt()
    s["dy"] = _normal(g, rows, cols, dt, pad, 1e-3)
    s["dh"] = _normal(g, rows, cols, dt, pad, 1e-3)
    s["dx"] = torch.empty((rows, cols), dtype=dt, device="cuda")
    s["dresidual"] = torch.empty((rows, cols), dtype=dt, device="cuda")
    s["dgamma"] = torch.empty(cols, device="cuda")
    return s


# ---- the plain forms

def _pcg(v):
    state = (v * 747796405 + 2891336453) & U32
    word = (((state >> ((state >> 28) + 4)) ^ state) * 277803737) & U32
    return (word >> 22) ^ word


def _dropped(v, p, seed):
    """Dropout of an FP32 tensor: element i is kept iff its 16 random bits reach p * 2^16."""
    if p == 0.0:
        return v
    key = _pcg(torch.tensor(seed >> 32, device="cuda"))
    key = _pcg(key ^ (seed & U32))
    pairs = _pcg(torch.arange((v.numel() + 1) // 2, device="cuda") ^ key)
    bits = torch.stack((pairs & 0xFFFF, pairs >> 16), 1).view(-1)[:v.numel()].view(v.shape)
    cut = int(round(p * 65536))
    return torch.where(bits >= cut, v * (65536.0 / (65536 - cut)), torch.zeros_like(v))


def _mx8(y):
    """E4M3 codes and UE8M0 scales of blocks of 32 along the rows: the smallest power of two
    under which no element of the block exceeds 448."""
    rows, cols = y.shape
    blocks = (cols + 31) // 32
    b = torch.nn.functional.pad(y, (0, blocks * 32 - cols)).view(rows, blocks, 32)
    m, ex = torch.frexp(b.abs().amax(2))
    e = torch.where(m <= 0.875, ex - 9, ex - 8)
    e = torch.where(m == 0, torch.full_like(e, -127), e.clamp(-127, 127))
    v = (b * torch.exp2(-e.float())[:, :, None]).clamp(-448.0, 448.0)
    codes = v.to(torch.float8_e4m3fn).view(rows, blocks * 32)[:, :cols].contiguous()
    return codes, (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)


def _plain(s):
    if s["op"] == "dropout":
        return _dropped(s["x"].float(), s["p"], s["seed"]).to(s["x"].dtype)
    if s["op"] == "norm":
        dt = s["x"].dtype
        h = s["residual"].float() + _dropped(s["x"].float(), s["p"], s["seed"])
        rstd = 1.0 / torch.sqrt((h * h).mean(1) + EPS)
        y = h * rstd[:, None] * s["gamma"].float()
        if s["out"] == "mx8":
            codes, scales = _mx8(y)
            return dict(h=h.to(dt), rstd=rstd, codes=codes, scales=scales)
        return dict(h=h.to(dt), rstd=rstd, y=y.to(dt))
    if s["op"] == "norm_back":
        dt = s["h"].dtype
        dy, rstd = s["dy"].float(), s["rstd"][:, None]
        n = s["h"].float() * rstd
        gy = dy * s["gamma"].float()
        g = s["dh"].float() + rstd * (gy - n * (gy * n).mean(1, keepdim=True))
        return dict(dresidual=g.to(dt), dx=_dropped(g, s["p"], s["seed"]).to(dt), dgamma=(dy * n).sum(0))
    x, w, labels = s["x"].float(), s["w"].float(), s["labels"]
    valid = (labels >= 0) & (labels < s["V"])
    at = torch.where(valid, labels, torch.zeros_like(labels))[:, None]
    logits = x @ w.t()
    top = logits.amax(1, keepdim=True)
    lse = top + torch.log(torch.exp(logits - top).sum(1, keepdim=True))
    loss = torch.where(valid, (lse - logits.gather(1, at))[:, 0], torch.zeros_like(lse[:, 0]))
    out = dict(loss=loss, lse=lse[:, 0])
    if s["train"]:
        d = torch.exp(logits.sub_(lse))
        d.scatter_add_(1, at, torch.full_like(lse, -1.0))
        d.mul_(torch.where(valid, s["dloss"], torch.zeros_like(s["dloss"]))[:, None])
        out["dx"] = (d @ w).to(torch.bfloat16)
        out["dw"] = (d.t() @ x).to(torch.bfloat16)
    return out


# ---- the library's entry points

def _library(s):
    import bit_microscaled_quantized_amd as nv
    code = nv.NVFP4_F32 if s.get("dt") == "f32" else nv.NVFP4_BF16
    if s["op"] == "dropout":
        x, y = s["x"], s["y"]
        nv.nvfp4_dropout(x, code, s["rows"], s["cols"], x.stride(0), s["p"], s["seed"], y, y.stride(0))
        return y
    if s["op"] == "norm":
        x, r, h, y = s["x"], s["residual"], s["h"], s.get("y")
        nv.nvfp4_rms_norm(x, r, code, s["rows"], s["cols"], x.stride(0), r.stride(0), s["gamma"], code, EPS,
                          s["p"], s["seed"], h, h.stride(0), y, s["cols"], s.get("codes"), s.get("scales"),
                          s["rstd"])
        if y is None:
            return dict(h=h, rstd=s["rstd"], codes=s["codes"], scales=s["scales"])
        return dict(h=h, rstd=s["rstd"], y=y)
    if s["op"] == "norm_back":
        dy, dh, h, dx, dr = s["dy"], s["dh"], s["h"], s["dx"], s["dresidual"]
        ws = torch.empty(nv.nvfp4_rms_norm_backward_workspace_size(s["rows"], s["cols"]), dtype=torch.uint8,
                         device="cuda")
        nv.nvfp4_rms_norm_backward(dy, dh, h, code, s["rows"], s["cols"], dy.stride(0), dh.stride(0), h.stride(0),
                                   s["gamma"], code, s["rstd"], s["p"], s["seed"], dx, dx.stride(0), dr,
                                   dr.stride(0), s["dgamma"], ws)
        return dict(dresidual=dr, dx=dx, dgamma=s["dgamma"])
    T, V, H, x, w = s["T"], s["V"], s["H"], s["x"], s["w"]
    ws = torch.empty(nv.nvfp4_linear_cross_entropy_workspace_size(T, V, H, s["train"]), dtype=torch.uint8,
                     device="cuda")
    nv.nvfp4_linear_cross_entropy(T, V, H, x, H, w, H, s["labels"], s["loss"], s["lse"], ws)
    out = dict(loss=s["loss"], lse=s["lse"])
    if s["train"]:
        nv.nvfp4_linear_cross_entropy_backward(T, V, H, x, H, w, H, s["labels"], s["lse"], s["dloss"], s["dx"], H,
                                               s["dw"], nv.NVFP4_BF16, H, 0.0, ws)
        out.update(dx=s["dx"], dw=s["dw"])
    return out


def run(state):
    return _library(state) if own else _plain(state)


def work(case):
    if case["op"] == "loss":
        T, V, H = case["T"], case["V"], case["H"]
        once = 2.0 * T * V * H  # one product of tokens, vocabulary and hidden size
        read = 2 * (T * H + V * H) + 8 * T
        if case["train"]:  # logits, gradient of the hidden states, gradient of the weight
            return dict(bytes=2 * read + 12 * T, flops=3 * once)
        return dict(bytes=read + 8 * T, flops=once)
    n, size = case["rows"] * case["cols"], 4 if case["dt"] == "f32" else 2
    if case["op"] == "dropout":
        return dict(bytes=2 * n * size, flops=2 * n)
    if case["op"] == "norm":
        held = n * size if case["out"] == "y" else n + case["rows"] * ((case["cols"] + 31) // 32)
        return dict(bytes=3 * n * size + held + case["cols"] * size + 4 * case["rows"], flops=6 * n)
    return dict(bytes=5 * n * size + case["cols"] * (size + 4) + 4 * case["rows"], flops=12 * n)


# ---- the definitions in 64 bits, written apart from the plain forms

def _keep64(n, p, seed):
    """Truth of `kept` per element index, from the hash's definition on 32-bit words held in int64."""
    def hashed(v):
        st = torch.remainder(v * 747796405 + 2891336453, 1 << 32)
        wd = torch.remainder(torch.bitwise_xor(torch.bitwise_right_shift(st, torch.bitwise_right_shift(st, 28) + 4), st)
                             * 277803737, 1 << 32)
        return torch.bitwise_xor(torch.bitwise_right_shift(wd, 22), wd)

    def scalar(v):
        return int(hashed(torch.tensor([v], dtype=torch.int64))[0])

    key = scalar((seed & U32) ^ scalar(seed >> 32))
    i = torch.arange(n, device="cuda", dtype=torch.int64)
    word = hashed(torch.bitwise_xor(torch.div(i, 2, rounding_mode="floor"), key))
    half = torch.where(torch.remainder(i, 2) == 1, torch.div(word, 65536, rounding_mode="floor"),
                       torch.remainder(word, 65536))
    return half >= round(p * 65536)


def _drop64(v, p, seed):
    if p == 0.0:
        return v
    kept = _keep64(v.numel(), p, seed).view(v.shape)
    cut = round(p * 65536)
    return torch.where(kept, v * 65536.0 / (65536 - cut), 0.0)


def _e4m3_64(v):
    """Nearest E4M3 value of |v| <= 448, ties to the even code, in float64."""
    mag = torch.log2(v.abs().clamp(min=2.0 ** -20)).floor().clamp(min=-6.0)
    step = torch.pow(2.0, mag - 3.0)
    return torch.round(v / step) * step  # torch.round takes ties to even


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "dropout":
        return _drop64(s["x"].double(), case["p"], s["seed"])
    if case["op"] == "norm":
        h = _drop64(s["x"].double(), case["p"], s["seed"]).add_(s["residual"].double())
        rstd = (torch.linalg.vecdot(h, h) / case["cols"] + EPS).pow(-0.5)
        y = torch.einsum("rc,r,c->rc", h, rstd, s["gamma"].double())
        if case["out"] == "y":
            return dict(h=h, rstd=rstd, y=y)
        short = -case["cols"] % 32
        blocks = torch.cat((y, y.new_zeros(case["rows"], short)), 1).unflatten(1, (-1, 32))
        top = blocks.abs().max(2).values
        e = torch.ceil(torch.log2(top / 448.0))
        e = torch.where(top > torch.pow(2.0, e) * 448.0, e + 1, e)
        e = torch.where(top <= torch.pow(2.0, e - 1) * 448.0, e - 1, e).clamp(-127, 127)
        scale = torch.pow(2.0, e)
        codes = _e4m3_64(blocks / scale[..., None]).flatten(1)[:, :case["cols"]]
        return dict(h=h, rstd=rstd, codes=codes, scales=scale)
    if case["op"] == "norm_back":
        dy, h, r = s["dy"].double(), s["h"].double(), s["rstd"].double()
        a = dy * s["gamma"].double()
        c = torch.linalg.vecdot(a, h) * r.pow(3) / case["cols"]
        g = s["dh"].double() + torch.einsum("rc,r->rc", a, r) - torch.einsum("rc,r->rc", h, c)
        return dict(dresidual=g, dx=_drop64(g, case["p"], s["seed"]),
                    dgamma=torch.einsum("rc,rc,r->c", dy, h, r))
    T, V = case["T"], case["V"]
    x, w, labels = s["x"].double(), s["w"].double(), s["labels"]
    z = torch.matmul(x, w.transpose(0, 1))
    lse = torch.logsumexp(z, 1)
    rows = torch.nonzero((labels >= 0) & (labels < V))[:, 0]
    loss = torch.zeros(T, dtype=torch.float64, device="cuda")
    loss[rows] = lse[rows] - z[rows, labels[rows]]
    out = dict(loss=loss, lse=lse)
    if case["train"]:
        z.sub_(lse[:, None]).exp_()
        z[rows, labels[rows]] -= 1.0
        weight = torch.zeros_like(loss)
        weight[rows] = s["dloss"][rows].double()
        z.mul_(weight[:, None])
        out["dx"] = torch.matmul(z, w)
        out["dw"] = torch.matmul(z.transpose(0, 1), x)
    return out
