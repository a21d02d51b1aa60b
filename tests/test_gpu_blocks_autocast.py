"""gated_act_linear under torch.autocast: its product is taken in the autocast type, as torch's
linear layer takes it, and the gradients come back in their tensors' types."""
import pytest

from tests import gpuio
from tests.test_gpu_blocks_layer import kept, plain_act, rnd

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,cast", [("float32", "bfloat16"), ("float32", "float16"), ("bfloat16", "float16"),
                                        ("bfloat16", "bfloat16")])
@pytest.mark.parametrize("inside", [False, True])
def test_gradients(dtype, cast, inside):
    """Against FP64 autograd at the kept values, relative in norm.  The product takes its factors in the autocast type and
    leaves in it, the gradients are rounded to their tensors' type: two factors and the result of each product, the
    upstream gradient's, and the leaf's, half a step each of the coarser type; FP32 sums below 200 terms.
    (FP16 factors are normal numbers here: magnitudes up to 2^4 that weigh in the norm above 2^-14.)"""
    torch = gpuio.torch_cuda()
    from bit_microscaled_quantized_amd.blocks import gated_act_linear
    t, c = getattr(torch, dtype), getattr(torch, cast)
    gate, up = (rnd(torch, i, 3, 50, 160, dtype=t).requires_grad_() for i in (1, 2))
    w = rnd(torch, 3, 96, 160, scale=0.1, dtype=t).requires_grad_()
    dz = rnd(torch, 4, 3, 50, 96, dtype=c)
    with torch.autocast("cuda", dtype=c):
        z = gated_act_linear(gate, up, w, "silu")
        assert z.dtype == c
        if inside:
            z.backward(dz)
    if not inside:
        z.backward(dz)
    ref = [kept(torch, v).double().requires_grad_() for v in (gate, up)] + [w.detach().double().requires_grad_()]
    (plain_act(torch, "silu", ref[0]) * ref[1] @ ref[2].t()).backward(dz.double())
    half = max(torch.finfo(t).eps, torch.finfo(c).eps) / 2
    for a, b in zip((gate, up, w), ref):
        assert a.grad.dtype == t and a.grad.shape == a.shape
        assert ((a.grad.double() - b.grad).norm() / b.grad.norm()).item() <= 5 * half + 200 * 2.0 ** -24


@pytest.mark.parametrize("leaf", [0, 1, 2])
def test_one_gradient_alone(leaf):
    torch = gpuio.torch_cuda()
    from bit_microscaled_quantized_amd.blocks import gated_act_linear
    tensors = [rnd(torch, 1, 40, 160), rnd(torch, 2, 40, 160), rnd(torch, 3, 96, 160, scale=0.1)]
    dz = rnd(torch, 4, 40, 96, dtype=torch.bfloat16)

    def grads(of):
        leaves = [v.clone().requires_grad_(i in of) for i, v in enumerate(tensors)]
        with torch.autocast("cuda", dtype=torch.bfloat16):
            z = gated_act_linear(*leaves, "gelu")
        z.backward(dz)
        return [v.grad for v in leaves]
    one = grads([leaf])
    assert [g is not None for g in one] == [i == leaf for i in range(3)]
    assert one[leaf].dtype == torch.float32 and torch.equal(one[leaf], grads([0, 1, 2])[leaf])
