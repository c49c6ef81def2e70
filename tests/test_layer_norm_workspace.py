"""The LayerNorm backward's workspace: bounded by the partial sums that fill the
GPU, whatever the width; and the gradients with fewer of them."""

import pytest
import torch

import diffusion_transformer_image_nvfp4_b200 as kl
from diffusion_transformer_image_nvfp4_b200 import build


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


def test_wide_rows_do_not_ask_for_more_than_the_partial_sums_need():
    size = kl.lib().kl_layer_norm_backward_workspace_size
    for dt in (0, 1, 2):
        for c in (1 << 14, 20000, 33000, (1 << 16) + 3, 1 << 20, 1 << 24):
            for g in (1, 2, 7, 148):
                n = size(dt, 700 * 148 * 14, c, g)
                one = (g * 2 * c * 4 + 255) // 256 * 256
                assert one <= n <= max(one, 20 << 20), (dt, c, g, n)
    # up to 16,384 columns a split for every SM
    assert size(0, 4096, 16384, 1) == 148 * 2 * 16384 * 4


@pytest.mark.gpu
@pytest.mark.parametrize("R,C,groups", [(600, 16384 + 8, 1), (450, 33001, 1), (302, 1 << 16, 2), (40, 1 << 18, 1),
                                        (9, 700001, 3)])
def test_gradients_of_wide_rows(R, C, groups):
    from tests.test_gpu_layer_norm import _params, _randn

    for dtype in (torch.bfloat16, torch.float32):
        x, dy = _randn((R, C), 1, dtype, 2.0, 1.0), _randn((R, C), 2, dtype)
        gain, bias = _params("modulate", groups, C, torch.float32, 3)
        _, mean, rstd = kl.layer_norm_forward(x, gain, bias, modulate=True)
        got = kl.layer_norm_backward(dy, x, mean, rstd, gain, modulate=True)
        _check_sums(got, dy, x, mean, rstd, groups)
        again = kl.layer_norm_backward(dy, x, mean, rstd, gain, modulate=True)
        assert all(torch.equal(a, b) for a, b in zip(got, again))
    assert kl.device_status() == "KL_OK"


def _check_sums(got, dy, x, mean, rstd, groups):
    """dgain and dbias: a thread adds at most the group's rows, in order, and the
    partial sums after them; each term has three roundings."""
    X, D = x.double(), dy.double()
    xh = (X - mean.double()[:, None]) * rstd.double()[:, None]
    shape = (groups, -1, X.shape[1])
    tol = (X.shape[0] // groups + 64) * 2.0 ** -24
    for a, t in ((got[1], D * xh), (got[2], D)):
        t = t.view(shape)
        assert ((a.double() - t.sum(1)).abs() <= tol * t.abs().sum(1) + 1e-37).all()
