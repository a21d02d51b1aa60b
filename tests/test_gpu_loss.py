"""The linear softmax cross entropy and its gradient against 64-bit computations.

Tolerances count roundings: u = 2^-24 (half a step of FP32), 2^-8 half a step of
BF16.  A logit is a sum of H products, within E = (H + 1) u sum |x w| in any
order; lse moves by at most the largest E of the row, plus the exponentials' and
additions' roundings, a few u each and one per joined part.  d = g (p - 1[label])
is rounded once to BF16 for the products, whose sums run over V or the tokens.
Values below the types' normal range, 2^-126, may come out as anything below it."""
import numpy as np
import pytest

import bit_microscaled_quantized_amd as nv
from tests import gpuio

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TINY = 2.0 ** -126
BF, F32 = nv.NVFP4_BF16, nv.NVFP4_F32


class Head:
    """One problem: device inputs (x, w with `pad` more columns a row, gaps NaN)
    and the 64-bit values."""

    def __init__(self, T, V, H, ignore, pad=0, seed=0, lean=True):
        torch = gpuio.torch_cuda()
        self.T, self.V, self.H, self.ld = T, V, H, H + pad
        g = torch.Generator(device="cuda").manual_seed(seed + T * 7 + V * 3 + H)
        rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")
        self.wb = torch.full((V, self.ld), float("nan"), dtype=torch.bfloat16, device="cuda")
        self.w = self.wb[:, :H]
        self.w.copy_(rnd(V, H) * (1.0 / H) ** 0.5)
        self.xb = torch.full((T, self.ld), float("nan"), dtype=torch.bfloat16, device="cuda")
        self.x = self.xb[:, :H]
        y = torch.randint(V, (T,), generator=g, device="cuda")
        x = rnd(T, H)
        if lean:
            x += 4 * torch.rand(T, 1, generator=g, device="cuda") * self.w[y].float()
        self.x.copy_(x)
        off = torch.rand(T, generator=g, device="cuda") < ignore
        bad = torch.tensor([-100, -1, V, V + 5, 2 ** 62, -2 ** 63], device="cuda")
        self.labels = torch.where(off, bad[torch.arange(T, device="cuda") % 6], y)
        self.valid = ~off
        self.dloss = rnd(T) / max(T, 1)
        self.torch = torch

    def reference(self):
        torch = self.torch
        x, w = self.x.double(), self.w.double()
        z = x @ w.t()
        mag = x.abs() @ w.abs().t()
        E = (self.H + 1) * U * (mag.amax(1) if self.T else mag.sum(1))
        lse = torch.logsumexp(z, 1)
        rows = torch.nonzero(self.valid)[:, 0]
        loss = torch.zeros_like(lse)
        loss[rows] = lse[rows] - z[rows, self.labels[rows]]
        p = torch.exp(z - lse[:, None])
        d = p.clone()
        d[rows, self.labels[rows]] -= 1
        g = torch.where(self.valid, self.dloss.double(), torch.zeros_like(lse))
        self.d = d * g[:, None]
        # error of d: the logit and lse (E each, and a few u of lse), exp, products; then BF16
        e = 2 * E + 64 * U * (1 + lse.abs())
        self.dd = g.abs()[:, None] * p * (e[:, None] + 8 * U) + self.d.abs() * 2.0 ** -8 + TINY
        self.xd, self.wd = x, w
        self.E, self.lse, self.loss = E, lse, loss
        return self

    def forward(self):
        torch = self.torch
        gd = gpuio.Guarded()
        loss, lse = gd.alloc((self.T,), torch.float32), gd.alloc((self.T,), torch.float32)
        n = nv.nvfp4_linear_cross_entropy_workspace_size(self.T, self.V, self.H, False)
        ws = gd.alloc((n // 4,), torch.float32, fill=float("nan"))
        nv.nvfp4_linear_cross_entropy(self.T, self.V, self.H, self.x, self.ld, self.w, self.ld, self.labels, loss, lse,
                                      ws)
        torch.cuda.synchronize()
        gd.check()
        return loss, lse

    def backward(self, lse, dw_dt=BF, beta=0.0, want=("dx", "dw"), dw0=None, out_pad=0, labels=None):
        torch = self.torch
        gd = gpuio.Guarded()
        ld = self.H + out_pad
        dx = gd.alloc((self.T, ld), torch.bfloat16, fill=7.0) if "dx" in want else None
        t = torch.bfloat16 if dw_dt == BF else torch.float32
        dw = None
        if "dw" in want:
            dw = gd.alloc((self.V, ld), t, fill=7.0)
            if dw0 is not None:
                dw[:, :self.H].copy_(dw0)
        n = nv.nvfp4_linear_cross_entropy_workspace_size(self.T, self.V, self.H, True)
        ws = gd.alloc((n // 4,), torch.float32, fill=float("nan"))
        nv.nvfp4_linear_cross_entropy_backward(self.T, self.V, self.H, self.x, self.ld, self.w, self.ld, self.labels,
                                               lse, self.dloss, dx, ld, dw, dw_dt, ld, beta, ws)
        torch.cuda.synchronize()
        gd.check()
        for o in (dx, dw):
            assert o is None or bool((o[:, self.H:] == 7.0).all()), "a gap between rows was written"
        return None if dx is None else dx[:, :self.H], None if dw is None else dw[:, :self.H]

    def check_forward(self, loss, lse):
        parts = (self.V + 127) // 128 + 256
        tol = self.E + U * (4 * self.lse.abs() + parts + 16)
        close(lse, self.lse, tol, "lse")
        close(loss, self.loss, 2 * tol + U * self.loss.abs(), "loss")
        assert bool((loss[~self.valid] == 0).all()), "ignored tokens have no loss"

    def check_dx(self, dx):
        ref = self.d @ self.wd
        tol = self.dd @ self.wd.abs() + (self.V + 64) * U * (self.d.abs() @ self.wd.abs()) + 2.0 ** -8 * ref.abs() + TINY
        close(dx, ref, tol * (1 + 2.0 ** -8), "dx")
        assert bool((dx[~self.valid] == 0).all()), "ignored tokens have no gradient"

    def check_dw(self, dw, dw_dt, dw0=None):
        ref, xa = self.d.t() @ self.xd, self.xd.abs()
        tol = self.dd.t() @ xa + (self.T + 64) * U * (self.d.abs().t() @ xa) + TINY
        if dw0 is not None:
            ref = ref + dw0.double()
        close(dw, ref, tol + (2.0 ** -8 if dw_dt == BF else 2 * U) * (ref.abs() + tol), "dw")


def close(got, ref, tol, what):
    bad = ~((got.double() - ref).abs() <= tol)
    if bool(bad.any()):
        i = tuple(bad.nonzero()[0].tolist())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {i}: {float(got[i])} for "
                             f"{float(ref[i])} +- {float(tol[i])}")


SHAPES = [(1, 1, 8), (1, 1000, 128), (3, 5, 16), (2, 64, 24), (15, 300, 72), (16, 1023, 264), (17, 129, 136),
          (33, 2000, 640), (48, 517, 1024), (64, 257, 64), (65, 1000, 200), (100, 33, 5120), (128, 128, 128),
          (130, 4099, 264), (255, 777, 1000), (256, 512, 512), (257, 1031, 512), (600, 1500, 72), (1030, 2050, 328)]


@pytest.mark.parametrize("T,V,H", SHAPES)
@pytest.mark.parametrize("ignore,pad", [(0.0, 0), (0.5, 8)])
def test_loss_and_gradients(T, V, H, ignore, pad):
    q = Head(T, V, H, ignore, pad).reference()
    loss, lse = q.forward()
    q.check_forward(loss, lse)
    dx, dw = q.backward(lse, out_pad=pad)
    q.check_dx(dx)
    q.check_dw(dw, BF)


@pytest.mark.parametrize("T,V,H", [(1, 30000, 64), (40, 70001, 40), (300, 70001, 64), (2500, 9001, 64)])
def test_large_vocabularies_and_many_tokens(T, V, H):
    q = Head(T, V, H, 0.3, seed=5).reference()
    loss, lse = q.forward()
    q.check_forward(loss, lse)
    dx, dw = q.backward(lse, dw_dt=F32)
    q.check_dx(dx)
    q.check_dw(dw, F32)


@pytest.mark.parametrize("T,ignore", [(1, 0.0), (5, 0.3), (16, 0.0), (17, 0.0), (32, 0.1), (33, 0.0), (64, 0.0), (65, 0.1),
                                      (300, 0.9), (2500, 0.98)])
@pytest.mark.parametrize("V,H", [(1031, 264), (40, 128)])
def test_few_labelled_tokens_keep_two_parts_of_d(T, ignore, V, H):
    """Up to 64 labelled tokens the products see d within 2^-16 of it (BF16, and the BF16
    of the rest: 2^-8 of 2^-8), so that FP32 dw and BF16 dx are that near."""
    q = Head(T, V, H, ignore, seed=21).reference()
    assert int(q.valid.sum()) <= 64
    _, lse = q.forward()
    dx, dw = q.backward(lse, F32)
    q.dd = q.dd - q.d.abs() * (2.0 ** -8 - 2.0 ** -16)
    q.check_dx(dx)
    q.check_dw(dw, F32)


@pytest.mark.parametrize("T", [100, 2500])
def test_a_shared_dloss_is_not_rounded(T):
    """Tokens of a mean loss whose labels the model gives little: d at the label is -dloss
    (1 - p), p < 2^-9, and held as -dloss, so dw there is within 2^-9 of dloss per token
    (and the sums' roundings), where BF16 of dloss = 1.0038 / 128 alone is off by 2^-8 of it."""
    q = Head(T, 2003, 128, 0.0, seed=2, lean=False)
    q.x.mul_(0.2)
    q.dloss.fill_(1.00387 / 128)
    q.reference()
    _, lse = q.forward()
    assert float((q.d.abs().amax(1) / q.dloss).min()) > 1 - 2.0 ** -9
    _, dw = q.backward(lse, F32)
    seen = q.torch.zeros(2003, dtype=q.torch.bool, device="cuda")
    seen[q.labels] = True
    ref = q.d.t() @ q.xd
    rel = float((dw.double() - ref)[seen].norm() / ref[seen].norm())
    assert rel < 2.0 ** -9, rel


def test_dloss_of_no_normal_size():
    """All zero: zero gradients.  Tiny or infinite: as products in FP32 give them."""
    q = Head(70, 300, 64, 0.0, seed=4).reference()
    torch = q.torch
    _, lse = q.forward()
    q.dloss.zero_()
    dx, dw = q.backward(lse, F32)
    assert bool((dx == 0).all()) and bool((dw == 0).all())
    q.dloss.fill_(1e-37)
    _, dw = q.reference().backward(lse, F32)
    assert float((dw.double() - q.d.t() @ q.xd).norm() / (q.d.t() @ q.xd).norm()) < 2.0 ** -7
    q.dloss[3] = float("inf")
    dx, dw = q.backward(lse, F32)
    assert bool((~dx[3].isfinite()).all()) and bool(dx[4:].isfinite().all())


def test_weight_rows_that_span_more_than_32_bits():
    """Vocabulary rows 2 MiB apart: from one piece's first row to its last is more than
    4 GiB, and some stages of the dx product end a few rows past that."""
    q = Head(3, 2300, 64, 0.0, pad=(1 << 20) - 64, seed=11).reference()
    loss, lse = q.forward()
    q.check_forward(loss, lse)
    dx, dw = q.backward(lse)
    q.check_dx(dx)
    q.check_dw(dw, BF)


@pytest.mark.parametrize("T,dw_dt,beta", [(3, BF, 0.0), (20, F32, 1.0), (60, BF, 1.0), (120, F32, 0.0), (300, BF, 0.0), (300, F32, 1.0),
                                          (1700, BF, 1.0)])
def test_weights_larger_than_the_caches(T, dw_dt, beta):
    """143 MB of weight, whose loads and gradient stores take other ways past the caches."""
    q = Head(T, 70001, 1024, 0.1, seed=13).reference()
    loss, lse = q.forward()
    q.check_forward(loss, lse)
    dw0 = None
    if beta:
        dw0 = (q.torch.randn(q.V, q.H, device="cuda") * 0.01).to(q.torch.bfloat16 if dw_dt == BF else q.torch.float32)
    dx, dw = q.backward(lse, dw_dt, beta, dw0=dw0)
    q.check_dx(dx)
    q.check_dw(dw, dw_dt, dw0)


@pytest.mark.parametrize("T", [1, 20, 90, 300])
@pytest.mark.parametrize("dw_dt", [BF, F32])
def test_accumulated_weight_gradient_and_single_outputs(T, dw_dt):
    V, H = 700, 192
    q = Head(T, V, H, 0.2, seed=3).reference()
    _, lse = q.forward()
    dw0 = q.torch.randn(V, H, device="cuda") * 0.01
    if dw_dt == BF:
        dw0 = dw0.bfloat16()
    dx, dw = q.backward(lse, dw_dt, 1.0, dw0=dw0)
    q.check_dw(dw, dw_dt, dw0)
    only_dx, none = q.backward(lse, dw_dt, want=("dx",))
    assert none is None and q.torch.equal(only_dx, dx)
    none, only_dw = q.backward(lse, dw_dt, 1.0, want=("dw",), dw0=dw0)
    assert none is None and q.torch.equal(only_dw, dw)


@pytest.mark.parametrize("T", [3, 70, 300])
def test_all_tokens_ignored(T):
    V, H = 400, 96
    q = Head(T, V, H, 1.1, seed=1).reference()
    loss, lse = q.forward()
    q.check_forward(loss, lse)
    dx, dw = q.backward(lse, F32)
    assert bool((dx == 0).all()) and bool((dw == 0).all()) and bool((loss == 0).all())
    dw0 = q.torch.randn(V, H, device="cuda")
    _, dw = q.backward(lse, F32, 1.0, dw0=dw0)
    assert q.torch.equal(dw, dw0)


def test_no_tokens():
    torch = gpuio.torch_cuda()
    V, H = 130, 24
    q = Head(0, V, H, 0.0)
    for dt, t in ((BF, torch.bfloat16), (F32, torch.float32)):
        dw = torch.full((V, H + 8), 7.0, dtype=t, device="cuda")
        args = (0, V, H, q.x, H, q.w, H, q.labels, q.dloss, q.dloss, None, 0, dw, dt, H + 8)
        nv.nvfp4_linear_cross_entropy_backward(*args, 1.0, None)
        assert bool((dw == 7).all())
        nv.nvfp4_linear_cross_entropy_backward(*args, 0.0, None)
        assert bool((dw[:, :H] == 0).all()) and bool((dw[:, H:] == 7).all())


@pytest.mark.parametrize("T", [12, 100, 520])
def test_ignored_tokens_may_hold_anything(T):
    """NaN in the ignored tokens' hidden states, lse and dloss reaches neither the
    other tokens nor the weight gradient: the values are those without them."""
    V, H = 300, 72
    q = Head(T, V, H, 0.5, seed=8).reference()
    loss, lse = q.forward()
    dx, dw = q.backward(lse, F32)
    nan = float("nan")
    q.x[~q.valid] = nan
    q.dloss[~q.valid] = nan
    loss2, lse2 = q.forward()
    ok = q.valid
    assert q.torch.equal(loss2, loss) and q.torch.equal(lse2[ok], lse[ok]) and bool(lse2[~ok].isnan().all())
    dx2, dw2 = q.backward(lse2, F32)
    assert q.torch.equal(dx2, dx) and q.torch.equal(dw2, dw)


@pytest.mark.parametrize("T", [2, 80, 300])
def test_wide_logits(T):
    """Logits of a few hundred: the running maximum keeps the exponentials in range."""
    q = Head(T, 900, 256, 0.0, seed=4, lean=False)
    q.x.mul_(60.0)
    q.reference()
    loss, lse = q.forward()
    assert float(lse.max()) > 100
    q.check_forward(loss, lse)
    dx, dw = q.backward(lse, F32)
    q.check_dx(dx)
    q.check_dw(dw, F32)


@pytest.mark.parametrize("T,V,H", [(1, 500, 64), (50, 3000, 256), (200, 3000, 256)])
def test_repeated_calls_agree_bit_for_bit(T, V, H):
    q = Head(T, V, H, 0.2, seed=6)
    a, b = q.forward(), q.forward()
    assert all(q.torch.equal(i, j) for i, j in zip(a, b))
    assert all(q.torch.equal(i, j) for i, j in zip(q.backward(a[1], F32), q.backward(a[1], F32)))


@pytest.mark.parametrize("T,V,H", [(5, 200, 64), (70, 300, 128)])
def test_gradient_against_differences(T, V, H):
    """<gradient, direction> against the central difference of sum dloss * loss in 64 bits."""
    q = Head(T, V, H, 0.3, seed=2).reference()
    torch = q.torch
    _, lse = q.forward()
    dx, dw = q.backward(lse, F32)
    g = torch.Generator(device="cuda").manual_seed(9)
    ex = torch.randn(T, H, generator=g, device="cuda").double()
    ew = torch.randn(V, H, generator=g, device="cuda").double()
    rows = torch.nonzero(q.valid)[:, 0]

    def value(s):
        z = (q.xd + s * ex) @ (q.wd + s * ew).t()
        return ((torch.logsumexp(z, 1)[rows] - z[rows, q.labels[rows]]) * q.dloss[rows].double()).sum()
    e = 1e-5
    diff = float((value(e) - value(-e)) / (2 * e))
    got = float((dx.double() * ex).sum() + (dw.double() * ew).sum())
    # BF16 roundings of d in both products and of dx, all counted at their largest
    size = float((q.d.abs() @ q.wd.abs() * ex.abs()).sum() * 2 + (q.d.abs().t() @ q.xd.abs() * ew.abs()).sum())
    assert abs(got - diff) <= size * 2.0 ** -8 + 1e-6 * abs(diff)
