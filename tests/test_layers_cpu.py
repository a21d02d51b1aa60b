"""Host-side checks of the operators between the quantized layers: every bad
argument is refused with the documented status before anything is enqueued,
workspace sizes need no device, and empty calls succeed without pointers."""
import ctypes

import pytest

import bit_microscaled_quantized_amd as nv
from bit_microscaled_quantized_amd import nvfp4 as b

FAKE = 1 << 20  # aligned, non-null, never dereferenced
NAN = float("nan")


def dropout(**kw):
    a = dict(x=FAKE, dt=0, rows=4, cols=40, ld_x=40, p=0.1, seed=1, y=FAKE, ld_y=40)
    a.update(kw)
    return nv.nvfp4_dropout(**a, stream=0, raise_on_error=False)


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), b.NVFP4_EINVAL),
    (dict(y=None), b.NVFP4_EINVAL),
    (dict(dt=2), b.NVFP4_EINVAL),
    (dict(dt=-1), b.NVFP4_EINVAL),
    (dict(p=-0.1), b.NVFP4_EINVAL),
    (dict(p=1.0), b.NVFP4_EINVAL),
    (dict(p=1.0 - 2.0 ** -18), b.NVFP4_EINVAL),   # rounds to dropping everything
    (dict(p=NAN), b.NVFP4_EINVAL),
    (dict(rows=-1), b.NVFP4_ESHAPE),
    (dict(cols=0), b.NVFP4_ESHAPE),
    (dict(ld_x=39), b.NVFP4_ESHAPE),
    (dict(ld_y=39), b.NVFP4_ESHAPE),
    (dict(ld_y=1 << 60), b.NVFP4_ESHAPE),
    (dict(rows=1 << 28, cols=1, ld_x=1, ld_y=1), b.NVFP4_ESHAPE),
    (dict(rows=(1 << 28) - 15, cols=1, ld_x=1, ld_y=1), b.NVFP4_ESHAPE),  # 2^32 lanes
    (dict(rows=1 << 20, cols=1 << 12, ld_x=1 << 12, ld_y=1 << 12), b.NVFP4_ESHAPE),  # 2^32 elements
    (dict(x=FAKE + 1), b.NVFP4_EALIGN),
    (dict(dt=1, y=FAKE + 2), b.NVFP4_EALIGN),
    (dict(rows=0, x=None, y=None), b.NVFP4_OK),
])
def test_dropout_arguments(kw, status):
    assert dropout(**kw) == status


def norm(**kw):
    a = dict(x=FAKE, residual=FAKE, dt=0, rows=4, cols=40, ld_x=40, ld_r=40, gamma=FAKE, gamma_dt=0, eps=1e-5,
             p=0.0, seed=0, h=FAKE, ld_h=40, y=FAKE, ld_y=40, codes=None, scales=None, rstd=FAKE)
    a.update(kw)
    return nv.nvfp4_rms_norm(**a, stream=0, raise_on_error=False)


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), b.NVFP4_EINVAL),
    (dict(gamma=None), b.NVFP4_EINVAL),
    (dict(y=None), b.NVFP4_EINVAL),                               # no output
    (dict(codes=FAKE, scales=FAKE), b.NVFP4_EINVAL),              # both outputs
    (dict(y=None, codes=FAKE), b.NVFP4_EINVAL),                   # codes without scales
    (dict(y=None, scales=FAKE), b.NVFP4_EINVAL),
    (dict(dt=3), b.NVFP4_EINVAL),
    (dict(gamma_dt=3), b.NVFP4_EINVAL),
    (dict(eps=-1e-5), b.NVFP4_EINVAL),
    (dict(eps=NAN), b.NVFP4_EINVAL),
    (dict(p=1.5), b.NVFP4_EINVAL),
    (dict(rows=-1), b.NVFP4_ESHAPE),
    (dict(cols=-1), b.NVFP4_ESHAPE),
    (dict(ld_x=39), b.NVFP4_ESHAPE),
    (dict(ld_r=39), b.NVFP4_ESHAPE),
    (dict(ld_h=39), b.NVFP4_ESHAPE),
    (dict(ld_y=39), b.NVFP4_ESHAPE),
    (dict(rows=1 << 16, cols=1 << 16, ld_x=1 << 16, ld_r=1 << 16, ld_h=1 << 16, ld_y=1 << 16), b.NVFP4_ESHAPE),
    (dict(residual=FAKE + 1), b.NVFP4_EALIGN),
    (dict(h=FAKE + 1), b.NVFP4_EALIGN),
    (dict(gamma_dt=1, gamma=FAKE + 2), b.NVFP4_EALIGN),
    (dict(rstd=FAKE + 2), b.NVFP4_EALIGN),
    (dict(rows=0, x=None, residual=None, gamma=None, h=None, y=None, rstd=None), b.NVFP4_OK),
])
def test_rms_norm_arguments(kw, status):
    assert norm(**kw) == status


def norm_back(**kw):
    a = dict(dy=FAKE, dh=FAKE, h=FAKE, dt=0, rows=4, cols=40, ld_dy=40, ld_dh=40, ld_h=40, gamma=FAKE, gamma_dt=0,
             rstd=FAKE, p=0.0, seed=0, dx=FAKE, ld_dx=40, dresidual=FAKE, ld_dr=40, dgamma=FAKE, workspace=FAKE,
             workspace_bytes=1 << 20)
    a.update(kw)
    return nv.nvfp4_rms_norm_backward(**a, stream=0, raise_on_error=False)


@pytest.mark.parametrize("kw,status", [
    (dict(dy=None), b.NVFP4_EINVAL),
    (dict(h=None), b.NVFP4_EINVAL),
    (dict(gamma=None), b.NVFP4_EINVAL),
    (dict(rstd=None), b.NVFP4_EINVAL),
    (dict(dx=None, dresidual=None, dgamma=None), b.NVFP4_EINVAL),
    (dict(workspace=None), b.NVFP4_EINVAL),
    (dict(workspace_bytes=16), b.NVFP4_ESHAPE),
    (dict(dt=2), b.NVFP4_EINVAL),
    (dict(p=-1.0), b.NVFP4_EINVAL),
    (dict(ld_dy=39), b.NVFP4_ESHAPE),
    (dict(ld_dh=39), b.NVFP4_ESHAPE),
    (dict(ld_h=39), b.NVFP4_ESHAPE),
    (dict(ld_dx=39), b.NVFP4_ESHAPE),
    (dict(ld_dr=39), b.NVFP4_ESHAPE),
    (dict(dy=FAKE + 1), b.NVFP4_EALIGN),
    (dict(dgamma=FAKE + 2), b.NVFP4_EALIGN),
    (dict(workspace=FAKE + 2), b.NVFP4_EALIGN),
])
def test_rms_norm_backward_arguments(kw, status):
    assert norm_back(**kw) == status


def test_rms_norm_backward_workspace():
    assert nv.nvfp4_rms_norm_backward_workspace_size(0, 5) == 0
    assert nv.nvfp4_rms_norm_backward_workspace_size(4, 40) > 0
    out = ctypes.c_int64(-7)
    f = b.load_library().nvfp4_rms_norm_backward_workspace_size
    assert f(-1, 40, ctypes.byref(out)) == b.NVFP4_ESHAPE and out.value == -7
    assert f(4, 40, None) == b.NVFP4_EINVAL
    with pytest.raises(nv.Nvfp4Error):
        nv.nvfp4_rms_norm_backward_workspace_size(4, 0)


BIG = 1 << 34


def loss(**kw):
    a = dict(T=4, V=100, H=64, x=FAKE, ld_x=64, w=FAKE, ld_w=64, labels=FAKE, loss=FAKE, lse=FAKE, workspace=FAKE,
             workspace_bytes=BIG)
    a.update(kw)
    return nv.nvfp4_linear_cross_entropy(**a, stream=0, raise_on_error=False)


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), b.NVFP4_EINVAL),
    (dict(w=None), b.NVFP4_EINVAL),
    (dict(labels=None), b.NVFP4_EINVAL),
    (dict(loss=None), b.NVFP4_EINVAL),
    (dict(lse=None), b.NVFP4_EINVAL),
    (dict(workspace=None), b.NVFP4_EINVAL),
    (dict(workspace_bytes=8), b.NVFP4_ESHAPE),
    (dict(T=-1), b.NVFP4_ESHAPE),
    (dict(V=0), b.NVFP4_ESHAPE),
    (dict(H=0), b.NVFP4_ESHAPE),
    (dict(H=60, ld_x=64, ld_w=64), b.NVFP4_ESHAPE),     # H must be a multiple of 8
    (dict(T=1 << 22), b.NVFP4_ESHAPE),
    (dict(V=1 << 24), b.NVFP4_ESHAPE),
    (dict(T=1 << 20, V=(1 << 17) + 1, workspace_bytes=1 << 60), b.NVFP4_ESHAPE),
    (dict(ld_x=56), b.NVFP4_ESHAPE),
    (dict(ld_w=56), b.NVFP4_ESHAPE),
    (dict(ld_x=68), b.NVFP4_EALIGN),
    (dict(ld_w=68), b.NVFP4_EALIGN),
    (dict(x=FAKE + 8), b.NVFP4_EALIGN),
    (dict(w=FAKE + 2), b.NVFP4_EALIGN),
    (dict(labels=FAKE + 4), b.NVFP4_EALIGN),
    (dict(loss=FAKE + 2), b.NVFP4_EALIGN),
    (dict(workspace=FAKE + 8), b.NVFP4_EALIGN),
    (dict(T=0, x=None, labels=None, loss=None, lse=None, workspace=None, workspace_bytes=0), b.NVFP4_OK),
])
def test_linear_cross_entropy_arguments(kw, status):
    assert loss(**kw) == status


def loss_back(**kw):
    a = dict(T=4, V=100, H=64, x=FAKE, ld_x=64, w=FAKE, ld_w=64, labels=FAKE, lse=FAKE, dloss=FAKE, dx=FAKE, ld_dx=64,
             dw=FAKE, dw_dt=0, ld_dw=64, beta=0.0, workspace=FAKE, workspace_bytes=BIG)
    a.update(kw)
    return nv.nvfp4_linear_cross_entropy_backward(**a, stream=0, raise_on_error=False)


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), b.NVFP4_EINVAL),
    (dict(lse=None), b.NVFP4_EINVAL),
    (dict(dloss=None), b.NVFP4_EINVAL),
    (dict(dx=None, dw=None), b.NVFP4_EINVAL),
    (dict(dw_dt=2), b.NVFP4_EINVAL),
    (dict(beta=0.5), b.NVFP4_EINVAL),
    (dict(beta=NAN), b.NVFP4_EINVAL),
    (dict(workspace=None), b.NVFP4_EINVAL),
    (dict(workspace_bytes=64), b.NVFP4_ESHAPE),
    (dict(H=4), b.NVFP4_ESHAPE),
    (dict(ld_dx=56), b.NVFP4_ESHAPE),
    (dict(ld_dw=56), b.NVFP4_ESHAPE),
    (dict(ld_dx=68), b.NVFP4_EALIGN),
    (dict(ld_dw=68), b.NVFP4_EALIGN),
    (dict(dw_dt=1, ld_dw=66), b.NVFP4_EALIGN),
    (dict(dx=FAKE + 8), b.NVFP4_EALIGN),
    (dict(dw=FAKE + 8), b.NVFP4_EALIGN),
    (dict(T=0, x=None, labels=None, lse=None, dloss=None, dx=None, dw=None, workspace=None, workspace_bytes=0),
     b.NVFP4_OK),
])
def test_linear_cross_entropy_backward_arguments(kw, status):
    assert loss_back(**kw) == status


def test_linear_cross_entropy_workspace():
    size = nv.nvfp4_linear_cross_entropy_workspace_size
    assert size(0, 10, 8, True) == 0
    for T, V, H in ((1, 1, 8), (257, 49999, 2048), (8192, 131072, 5120)):
        assert 0 < size(T, V, H, False) <= size(T, V, H, True)
    # the logits are not kept: the largest workspace is far below the logits' size in FP32
    assert size(8192, 131072, 5120, True) < 4 * 8192 * 131072 / 2
    out = ctypes.c_int64(-7)
    f = b.load_library().nvfp4_linear_cross_entropy_workspace_size
    assert f(4, 10, 12, 0, ctypes.byref(out)) == b.NVFP4_ESHAPE and out.value == -7
    assert f(4, 10, 8, 0, None) == b.NVFP4_EINVAL


def test_errors_raise_in_checked_mode():
    with pytest.raises(nv.Nvfp4Error) as e:
        nv.nvfp4_dropout(FAKE, 0, 4, 40, 40, 2.0, 0, FAKE, 40, stream=0)
    assert e.value.status == b.NVFP4_EINVAL


def test_autograd_layer_refuses_host_tensors_and_wrong_shapes():
    import torch
    from bit_microscaled_quantized_amd import layers
    x, w, y = torch.ones(4, 64).bfloat16(), torch.ones(10, 64).bfloat16(), torch.zeros(4, dtype=torch.int64)
    g = torch.ones(64).bfloat16()
    with pytest.raises(ValueError, match="GPU"):
        layers.dropout(x, 0.1, 1)
    with pytest.raises(ValueError, match="GPU"):
        layers.add_rms_norm(x, x, g)
    with pytest.raises(ValueError, match="GPU"):
        layers.rms_norm_mx8(x, x, g)
    with pytest.raises(ValueError, match="GPU"):
        layers.linear_cross_entropy(x, w, y)
