"""The projection path records no autograd graph: a tensor that requires a
gradient is refused while grad mode is on, by every call and in every place
(checked before anything that needs a GPU)."""

import pytest
import torch

import diffusion_transformer_image_nvfp4_b200 as kl
from diffusion_transformer_image_nvfp4_b200 import build


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


def _leaf(*shape):
    return torch.zeros(*shape, requires_grad=True)


BY_X = {
    "encode": lambda x: kl.quantize_fp8_block(x),
    "rotary": lambda x: kl.rope_axes(x.view(4, 2, 8), torch.zeros(4, 1), (4,)),
    "layer norm": lambda x: kl.layer_norm_forward(x),
    "layer norm backward": lambda x: kl.layer_norm_backward(x, x.detach(), torch.zeros(4), torch.zeros(4)),
}


@pytest.mark.parametrize("call", BY_X.values(), ids=BY_X)
def test_a_tensor_that_requires_a_gradient_is_refused(call):
    x = _leaf(4, 16)
    for t in (x, x * 2, torch.nn.Parameter(torch.zeros(4, 16))):
        with pytest.raises(ValueError, match="requires a gradient"):
            call(t)
    # not where no graph is recorded: these go on to ask for CUDA tensors
    for quiet in (torch.no_grad, torch.inference_mode):
        with quiet(), pytest.raises(ValueError, match="CUDA"):
            call(x)
    with pytest.raises(ValueError, match="CUDA"):
        call(x.detach())

    class Call(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x):
            return call(x)

    with pytest.raises(ValueError, match="CUDA"):
        Call.apply(x)
