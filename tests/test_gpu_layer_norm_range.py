"""kl_layer_norm_backward near the ends of fp32's range, in every kernel that
many rows can take: 16-byte vectors (one to three a thread), pairs and single
elements, with and without columns that the last threads have no work for."""

import pytest
import torch

import diffusion_transformer_image_nvfp4_b200 as kl
from tests.test_gpu_layer_norm import _check_backward, _params, _randn

pytestmark = pytest.mark.gpu

WIDTHS = [256, 258, 1000, 1003, 1026, 2000, 2047, 3080]


@pytest.mark.parametrize("C", WIDTHS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("spread,grad,eps", [(1e15, 1e25, 1e-6), (1e-15, 1e-30, 0.0)])
def test_spreads_whose_product_with_the_gradient_leaves_the_range(C, dtype, spread, grad, eps):
    # dy (x - mean) is 1e40 or 1e-45 here, dy xhat and every result are not
    for R in (1203, 5):
        x, dy = _randn((R, C), C, dtype, spread, spread), _randn((R, C), C + 1, dtype, grad)
        gain, _ = _params("gain", 1, C, torch.float32, 3)
        _, mean, rstd = kl.layer_norm_forward(x, gain, eps=eps)
        got = kl.layer_norm_backward(dy, x, mean, rstd, gain)
        assert all(torch.isfinite(t).all() for t in got)
        _check_backward(got, dy, x, mean, rstd, gain, False, 1)
        dx = kl.layer_norm_backward(dy, x, mean, rstd, gain, param_grads=False)[0]
        _check_backward((dx, None, None), dy, x, mean, rstd, gain, False, 1)


@pytest.mark.parametrize("C", WIDTHS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_columns_past_the_last_take_no_part(C, dtype):
    # rows for which 0 in place of a value would give xhat = -2^150: not finite
    R = 1203
    x, dy = _randn((R, C), C, dtype, 1.0), _randn((R, C), C + 1, dtype)
    _, mean, rstd = kl.layer_norm_forward(x)
    for r in (0, 7, 600, R - 1):
        x[r], mean[r], rstd[r] = 2.0 ** 100, 2.0 ** 100, 2.0 ** 50
    got = kl.layer_norm_backward(dy, x, mean, rstd)
    assert all(torch.isfinite(t).all() for t in got)
    _check_backward(got, dy, x, mean, rstd, None, False, 1)
