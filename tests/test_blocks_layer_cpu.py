"""What the layer over the operators of a residual block in eight bits refuses before any
kernel is called: host tensors, and tensors on another device than the current one."""
import pytest
import torch

from bit_microscaled_quantized_amd import blocks


def calls(x, g):
    w = x[:1]
    c = x.to(torch.int8)
    return {
        "block_norms": lambda: blocks.block_norms(x, x, g, g),
        "block_norms_int8": lambda: blocks.block_norms_int8(x, x, g, g),
        "gated_act": lambda: blocks.gated_act(x, x),
        "gated_act_linear": lambda: blocks.gated_act_linear(x, x, w),
        "keep8": lambda: blocks.keep8(x),
        "restore8": lambda: blocks.restore8(c, c.view(torch.uint8)[:, :2]),
        "int8_quantize": lambda: blocks.int8_quantize(x),
        "int8_quantize_gated": lambda: blocks.int8_quantize_gated(x, x),
        "int8_matmul": lambda: blocks.int8_matmul(c, g[:4], c, g[:4]),
        "Int8Linear": lambda: blocks.Int8Linear(x),
    }


@pytest.mark.parametrize("name", sorted(calls(torch.ones(4, 64), torch.ones(64))))
def test_host_tensors_are_refused(name):
    with pytest.raises(ValueError, match="GPU"):
        calls(torch.ones(4, 64), torch.ones(64))[name]()


class Elsewhere(torch.Tensor):
    """A tensor that says it is on a device that is not the current one."""
    is_cuda = True

    @property
    def device(self):
        return torch.device("cuda", 1)


@pytest.mark.parametrize("name", ["gated_act", "keep8", "int8_quantize"])
def test_tensors_on_another_device_are_refused(name, monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    x = torch.ones(4, 64).as_subclass(Elsewhere)
    with pytest.raises(ValueError, match="current device"):
        calls(x, torch.ones(64))[name]()


def test_unknown_activations_are_refused():
    for call in (blocks.gated_act, blocks.int8_quantize_gated):
        with pytest.raises(ValueError, match="act"):
            call(torch.ones(4, 64), None, "swish")
