"""Host-side checks of the operators of a residual block in eight bits: every bad
argument is refused with the documented status before anything is enqueued,
workspace sizes need no device, and empty calls succeed without pointers."""
import ctypes

import pytest

import bit_microscaled_quantized_amd as nv
from bit_microscaled_quantized_amd import nvfp4 as b

FAKE = 1 << 20  # aligned, non-null, never dereferenced
NAN, INF = float("nan"), float("inf")
E, S, A, OK = b.NVFP4_EINVAL, b.NVFP4_ESHAPE, b.NVFP4_EALIGN, b.NVFP4_OK
HUGE = 1 << 60


def quantize(**kw):
    a = dict(x=FAKE, dt=0, rows=4, cols=40, ld_x=40, codes=FAKE, ld_codes=48, scales=FAKE)
    a.update(kw)
    return nv.nvfp4_int8_quantize(**a, stream=0, raise_on_error=False)


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), E), (dict(codes=None), E), (dict(scales=None), E), (dict(dt=2), E), (dict(dt=-1), E),
    (dict(rows=-1), S), (dict(cols=0), S), (dict(ld_x=39), S), (dict(ld_codes=32), S), (dict(ld_x=HUGE), S),
    (dict(rows=1, cols=1 << 31, ld_x=1 << 31, ld_codes=1 << 31), S),
    (dict(rows=1 << 20, cols=1 << 12, ld_x=1 << 12, ld_codes=1 << 12), S),
    (dict(rows=(1 << 28) - 15, cols=1, ld_x=1, ld_codes=16), S),
    (dict(ld_codes=40), A), (dict(ld_codes=56), A), (dict(codes=FAKE + 8), A), (dict(scales=FAKE + 2), A),
    (dict(x=FAKE + 1), A), (dict(dt=1, x=FAKE + 2), A),
    (dict(rows=0, x=None, codes=None, scales=None), OK),
])
def test_int8_quantize_arguments(kw, status):
    assert quantize(**kw) == status


def quantize_gated(**kw):
    a = dict(act=1, gate=FAKE, up=FAKE, dt=0, rows=4, cols=40, ld_gate=40, ld_up=40, codes=FAKE, ld_codes=48, scales=FAKE)
    a.update(kw)
    return nv.nvfp4_int8_quantize_gated(**a, stream=0, raise_on_error=False)


@pytest.mark.parametrize("kw,status", [
    (dict(act=4), E), (dict(act=-1), E), (dict(gate=None), E), (dict(codes=None), E), (dict(scales=None), E),
    (dict(dt=7), E), (dict(ld_gate=39), S), (dict(ld_up=39), S), (dict(up=FAKE + 1), A), (dict(gate=FAKE + 1), A),
    (dict(rows=0, gate=None, up=None, codes=None, scales=None), OK),
])
def test_int8_quantize_gated_arguments(kw, status):
    assert quantize_gated(**kw) == status


def gemm(**kw):
    a = dict(M=4, N=40, K=64, a=FAKE, lda=64, a_scales=FAKE, b=FAKE, ldb=64, b_scales=FAKE, c=FAKE, c_dt=0, ldc=40,
             workspace=FAKE, workspace_bytes=1 << 40)
    a.update(kw)
    return nv.nvfp4_int8_gemm(**a, stream=0, raise_on_error=False)


@pytest.mark.parametrize("kw,status", [
    (dict(a=None), E), (dict(a_scales=None), E), (dict(b=None), E), (dict(b_scales=None), E), (dict(c=None), E),
    (dict(c_dt=2), E),
    (dict(M=-1), S), (dict(N=0), S), (dict(K=0), S), (dict(K=8), S), (dict(K=72, lda=80, ldb=80), S),
    (dict(K=131072, lda=131072, ldb=131072), S),  # 128 * 128 * K reaches 2^31
    (dict(M=1 << 24), S), (dict(N=1 << 24, ldc=1 << 24), S), (dict(M=1 << 20, N=(1 << 15) + 1, ldc=1 << 17), S),
    (dict(lda=48), S), (dict(ldb=48), S), (dict(ldc=39), S), (dict(lda=1 << 23), S), (dict(ldb=1 << 23), S),
    (dict(ldc=HUGE), S),
    (dict(lda=72), A), (dict(ldb=72), A), (dict(a=FAKE + 8), A), (dict(b=FAKE + 8), A), (dict(a_scales=FAKE + 2), A),
    (dict(b_scales=FAKE + 2), A), (dict(c=FAKE + 1), A), (dict(c_dt=1, c=FAKE + 2), A), (dict(workspace=FAKE + 8), A),
    (dict(M=0, a=None, a_scales=None, b=None, b_scales=None, c=None, workspace=None), OK),
])
def test_int8_gemm_arguments(kw, status):
    assert gemm(**kw) == status


def test_int8_gemm_workspace():
    size = nv.nvfp4_int8_gemm_workspace_size
    assert size(0, 5, 16) == 0 and size(8192, 20480, 5120) == 0
    for M, N, K in ((1, 1, 16), (17, 20480, 5120), (300, 513, 131056), ((1 << 24) - 1, 1, 16), (1, (1 << 24) - 1, 16),
                    (1 << 20, 1 << 15, 16), (1 << 20, 1 << 15, 131056)):
        assert 0 <= size(M, N, K) <= 1 << 28 and size(M, N, K) % 16 == 0
    out = ctypes.c_int64(-7)
    f = b.load_library().nvfp4_int8_gemm_workspace_size
    assert f(4, 4, 17, ctypes.byref(out)) == S and out.value == -7
    assert f(4, 4, 16, None) == E
    with pytest.raises(nv.Nvfp4Error):
        size(4, 0, 16)


def norms(**kw):
    a = dict(x=FAKE, residual=FAKE, gate=FAKE, dt=0, rows=4, cols=40, ld_x=40, ld_r=40, ld_gate=40, gate_act=0,
             post_gamma=FAKE, pre_gamma=FAKE, gamma_dt=0, eps=1e-5, scale=1.0, h=FAKE, ld_h=40, y=FAKE, ld_y=40,
             codes=None, ld_codes=0, scales=None, post_rstd=FAKE, pre_rstd=FAKE)
    a.update(kw)
    return nv.nvfp4_block_norms(**a, stream=0, raise_on_error=False)


CODES = dict(y=None, codes=FAKE, ld_codes=48, scales=FAKE)


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), E), (dict(post_gamma=None), E), (dict(pre_gamma=None), E), (dict(y=None), E),
    (dict(codes=FAKE, scales=FAKE, ld_codes=48), E),  # both outputs
    (dict(y=None, codes=FAKE, ld_codes=48), E), (dict(y=None, scales=FAKE), E),
    (dict(dt=2), E), (dict(gamma_dt=2), E), (dict(gate_act=2), E), (dict(gate_act=-1), E), (dict(eps=-1.0), E),
    (dict(eps=NAN), E), (dict(scale=NAN), E), (dict(scale=INF), E),
    (dict(rows=-1), S), (dict(cols=0), S), (dict(ld_x=39), S), (dict(ld_r=39), S), (dict(ld_gate=39), S),
    (dict(ld_gate=-40), S), (dict(ld_h=39), S), (dict(ld_y=39), S), (dict(CODES, ld_codes=32), S),
    (dict(CODES, ld_codes=40), A), (dict(CODES, codes=FAKE + 4), A), (dict(CODES, scales=FAKE + 2), A),
    (dict(x=FAKE + 1), A), (dict(residual=FAKE + 1), A), (dict(gate=FAKE + 1), A), (dict(h=FAKE + 1), A),
    (dict(y=FAKE + 1), A), (dict(gamma_dt=1, post_gamma=FAKE + 2), A), (dict(gamma_dt=1, pre_gamma=FAKE + 2), A),
    (dict(post_rstd=FAKE + 2), A), (dict(pre_rstd=FAKE + 2), A),
    (dict(rows=0, x=None, residual=None, gate=None, post_gamma=None, pre_gamma=None, h=None, y=None, post_rstd=None,
          pre_rstd=None), OK),
])
def test_block_norms_arguments(kw, status):
    assert norms(**kw) == status


def norms_back(**kw):
    a = dict(dy=FAKE, dh=FAKE, h=FAKE, x=FAKE, gate=FAKE, dt=0, rows=4, cols=40, ld_dy=40, ld_dh=40, ld_h=40, ld_x=40,
             ld_gate=40, gate_act=0, post_gamma=FAKE, pre_gamma=FAKE, gamma_dt=0, post_rstd=FAKE, pre_rstd=FAKE,
             scale=1.0, dx=FAKE, ld_dx=40, dresidual=FAKE, ld_dr=40, dgate=FAKE, ld_dgate=40, dpost_gamma=FAKE,
             dpre_gamma=FAKE, workspace=FAKE, workspace_bytes=1 << 20)
    a.update(kw)
    return nv.nvfp4_block_norms_backward(**a, stream=0, raise_on_error=False)


@pytest.mark.parametrize("kw,status", [
    (dict(dy=None), E), (dict(h=None), E), (dict(x=None), E), (dict(post_gamma=None), E), (dict(pre_gamma=None), E),
    (dict(post_rstd=None), E), (dict(pre_rstd=None), E), (dict(gate=None), E),  # a dgate without a gate
    (dict(dx=None, dresidual=None, dgate=None, dpost_gamma=None, dpre_gamma=None), E),
    (dict(dt=2), E), (dict(gamma_dt=2), E), (dict(gate_act=3), E), (dict(scale=INF), E), (dict(workspace=None), E),
    (dict(workspace_bytes=16), S), (dict(rows=-1), S), (dict(cols=0), S), (dict(ld_dy=39), S), (dict(ld_dh=39), S),
    (dict(ld_h=39), S), (dict(ld_x=39), S), (dict(ld_gate=39), S), (dict(ld_dgate=39), S), (dict(ld_dx=39), S),
    (dict(ld_dr=39), S),
    (dict(dy=FAKE + 1), A), (dict(dh=FAKE + 1), A), (dict(h=FAKE + 1), A), (dict(x=FAKE + 1), A),
    (dict(gate=FAKE + 1), A), (dict(dx=FAKE + 1), A), (dict(dresidual=FAKE + 1), A), (dict(dgate=FAKE + 1), A),
    (dict(ld_gate=0, dgate=FAKE + 2), A), (dict(dpost_gamma=FAKE + 2), A), (dict(dpre_gamma=FAKE + 2), A),
    (dict(gamma_dt=1, pre_gamma=FAKE + 2), A), (dict(post_rstd=FAKE + 2), A), (dict(workspace=FAKE + 2), A),
    (dict(rows=0, dy=None, dh=None, h=None, x=None, gate=None, post_gamma=None, pre_gamma=None, post_rstd=None,
          pre_rstd=None, dx=None, dresidual=None, dgate=None, dpost_gamma=None, dpre_gamma=None, workspace=None,
          workspace_bytes=0), OK),
])
def test_block_norms_backward_arguments(kw, status):
    assert norms_back(**kw) == status


def test_block_norms_backward_workspace():
    size = nv.nvfp4_block_norms_backward_workspace_size
    assert size(0, 5) == 0 and size(4, 40) > 0
    f = b.load_library().nvfp4_block_norms_backward_workspace_size
    out = ctypes.c_int64(-7)
    assert f(-1, 40, ctypes.byref(out)) == S and out.value == -7
    assert f(4, 40, None) == E


def act(**kw):
    a = dict(act=1, gate=FAKE, up=FAKE, dt=0, rows=4, cols=40, ld_gate=40, ld_up=40, y=FAKE, ld_y=40, gate_codes=FAKE,
             gate_scales=FAKE, up_codes=FAKE, up_scales=FAKE)
    a.update(kw)
    return nv.nvfp4_gated_act(**a, stream=0, raise_on_error=False)


@pytest.mark.parametrize("kw,status", [
    (dict(act=4), E), (dict(act=-1), E), (dict(gate=None), E), (dict(dt=2), E),
    (dict(gate_scales=None), E), (dict(up_codes=None), E), (dict(up=None), E),       # codes of no up
    (dict(up_codes=None, up_scales=None), E),                                        # an up without codes
    (dict(gate_codes=None, gate_scales=None), E),                                    # up's codes alone
    (dict(up=None, y=None, gate_codes=None, gate_scales=None, up_codes=None, up_scales=None), E),  # no output
    (dict(rows=-1), S), (dict(cols=0), S), (dict(ld_gate=39), S), (dict(ld_up=39), S), (dict(ld_y=39), S),
    (dict(rows=1 << 28, cols=1), S), (dict(gate=FAKE + 1), A), (dict(up=FAKE + 1), A), (dict(dt=1, y=FAKE + 2), A),
    (dict(rows=0, gate=None, up=None, y=None, gate_codes=None, gate_scales=None, up_codes=None, up_scales=None), OK),
])
def test_gated_act_arguments(kw, status):
    assert act(**kw) == status


def act_back(**kw):
    a = dict(act=1, gate_codes=FAKE, gate_scales=FAKE, up_codes=FAKE, up_scales=FAKE, dy=FAKE, dt=0, rows=4, cols=40,
             ld_dy=40, dgate=FAKE, ld_dgate=40, dup=FAKE, ld_dup=40, y=FAKE, ld_y=40)
    a.update(kw)
    return nv.nvfp4_gated_act_backward(**a, stream=0, raise_on_error=False)


@pytest.mark.parametrize("kw,status", [
    (dict(act=9), E), (dict(gate_codes=None), E), (dict(gate_scales=None), E), (dict(up_scales=None), E), (dict(dt=-1), E),
    (dict(gate_codes=None, gate_scales=None), E), (dict(up_codes=None, up_scales=None), E),  # dup without up
    (dict(dy=None), E), (dict(dgate=None, dup=None), E),                                     # a dy for y alone
    (dict(dy=None, dgate=None, dup=None, y=None), E),
    (dict(rows=-1), S), (dict(cols=0), S), (dict(ld_dy=39), S), (dict(ld_dgate=39), S), (dict(ld_dup=39), S),
    (dict(ld_y=39), S), (dict(dy=FAKE + 1), A), (dict(dgate=FAKE + 1), A), (dict(dup=FAKE + 1), A), (dict(y=FAKE + 1), A),
    (dict(rows=0, gate_codes=None, gate_scales=None, up_codes=None, up_scales=None, dy=None, dgate=None, dup=None,
          y=None), OK),
])
def test_gated_act_backward_arguments(kw, status):
    assert act_back(**kw) == status
