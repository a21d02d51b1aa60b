"""Host-side refusals of the NVFP4 linear layer: nothing is launched on tensors that the
current device does not hold."""
import pytest
import torch

from bit_microscaled_quantized_amd import module


class Launched(Exception):
    pass


@pytest.fixture
def no_launch(monkeypatch):
    def fail(*args, **kw):
        raise Launched
    for name in ("nvfp4_quantize", "nvfp4_quantize_row_rht", "nvfp4_gemm", "nvfp4_gemm_bf16"):
        monkeypatch.setattr(module.nv, name, fail)


def test_host_tensors_are_refused(no_launch):
    x, w = torch.ones(64, 64).bfloat16(), torch.ones(64, 64).bfloat16()
    with pytest.raises(ValueError, match="GPU"):
        module.nvfp4_linear(x, w, 0, 1, 2)


def test_tensors_on_another_device_than_the_current_one_are_refused(no_launch, monkeypatch):
    """A tensor that says it is on GPU 1 while GPU 0 is current."""
    class Elsewhere(torch.Tensor):
        is_cuda = property(lambda self: True)
        device = property(lambda self: torch.device("cuda", 1))

    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    x = torch.ones(64, 64).bfloat16().as_subclass(Elsewhere)
    with pytest.raises(ValueError, match="cuda:0, got one on cuda:1"):
        module._function().forward(None, x, x, 0, 1, 2)
