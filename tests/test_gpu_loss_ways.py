"""The ways that the linear cross entropy takes for larger sizes, each at a size that takes
it: more than 4096 tokens, a vocabulary in several pieces, 256 x 256, 128 x 128 and 64 x 64 tiles where
the hidden size is no multiple of 128, few labelled tokens among many, and weights and
weight gradients on both sides of the caches' size.  References and tolerances are those of
test_gpu_loss: 64 bits, roundings counted."""
import pytest

from tests.test_gpu_loss import BF, F32, Head

pytestmark = pytest.mark.gpu


def check(T, V, H, ignore, dw_dt, beta=0.0, seed=31):
    q = Head(T, V, H, ignore, seed=seed).reference()
    loss, lse = q.forward()
    q.check_forward(loss, lse)
    dw0 = None
    if beta:
        dw0 = (q.torch.randn(V, H, device="cuda") * 0.01).to(q.torch.bfloat16 if dw_dt == BF else q.torch.float32)
    dx, dw = q.backward(lse, dw_dt, beta, dw0=dw0)
    q.check_dx(dx)
    q.check_dw(dw, dw_dt, dw0)
    return q


@pytest.mark.parametrize("T,V,H,ignore,dw_dt", [
    (4734, 6415, 288, 0.1, BF),       # listed and gathered by kernels of their own; 256 x 256 tiles, H = 288
    (5000, 1031, 264, 0.5, F32),
    (4097, 130, 64, 0.0, F32),
    (1944, 45515, 136, 0.5, BF),      # dx in 256 x 256 tiles and 16 or more parts
    (145, 54406, 208, 0.0, F32),
    (577, 35044, 152, 0.5, BF),       # dw in 256 x 256 tiles, inside the caches
    (529, 32919, 136, 0.0, F32),
    (541, 87205, 424, 0.3, F32),      # and beyond them
    (33, 40624, 136, 0.0, BF),        # dw in 128 x 128 tiles of one buffer, inside the caches
])
def test_many_tokens_and_large_tiles(T, V, H, ignore, dw_dt):
    check(T, V, H, ignore, dw_dt)


@pytest.mark.parametrize("T,V,H,ignore", [(4200, 1031, 264, 0.99), (76, 36650, 144, 0.9), (84, 49895, 128, 0.5),
                                          (160, 52900, 208, 0.9), (132, 50301, 256, 0.9), (68, 44852, 1600, 0.2),
                                          (69, 78679, 896, 0.2)])
def test_few_labelled_tokens_in_larger_tiles(T, V, H, ignore):
    """Up to 64 labelled tokens among more: two parts of d from one 128 x 128 or 256 x 256 tile."""
    q = check(T, V, H, ignore, BF)
    assert 0 < int(q.valid.sum()) <= 64


@pytest.mark.parametrize("T,V,H,ignore,dw_dt", [
    (1, 22866, 3008, 0.0, BF),        # the weight is read past the caches, H no multiple of 128
    (1, 65634, 512, 0.0, F32),        # and dw written past them
    (17, 30552, 2368, 0.0, BF),
    (74, 59930, 1344, 0.0, BF),
])
def test_few_tokens_over_large_weights(T, V, H, ignore, dw_dt):
    check(T, V, H, ignore, dw_dt)


@pytest.mark.parametrize("T,V,H,dw_dt,beta", [
    (3577, 75922, 128, F32, 0.0),     # pieces of 74752 rows; the last has fewer of 128 than dx has parts
    (3577, 75922, 128, BF, 1.0),
    (4000, 70001, 136, BF, 0.0),      # pieces of 65536
    (2509, 106348, 136, F32, 1.0),    # dx in 256 x 256 tiles
    (5001, 131072, 64, BF, 0.0),      # three pieces
])
def test_a_vocabulary_in_pieces(T, V, H, dw_dt, beta):
    """dx is added over the pieces, labels and dw's rows lie in all of them."""
    piece = (512 << 20) // (2 * ((T + 127) // 128 * 128)) // 256 * 256  # d of a piece in 512 MiB
    assert piece < V
    q = check(T, V, H, 0.2, dw_dt, beta)
    for v0 in range(0, V, piece):
        assert bool(((q.labels >= v0) & (q.labels < min(V, v0 + piece))).any())
