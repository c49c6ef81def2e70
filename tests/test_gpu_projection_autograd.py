"""The projection path's calls beside torch's autograd: what they write in place
is seen by it."""

import pytest
import torch

import diffusion_transformer_image_nvfp4_b200 as kl

pytestmark = pytest.mark.gpu


def _randn(*shape):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(sum(shape))).cuda()


def _rotate_in_place(t):
    pos = torch.arange(t.shape[0], dtype=torch.int32, device="cuda")[:, None]
    h = t.view(t.shape[0], 2, -1)
    kl.rope_axes(h, pos, (4,), out=h)


def _product_in_place(t):
    w = kl.quantize_fp8_block(_randn(t.shape[1], 32))
    kl.gemm_fp8_block(kl.quantize_fp8_block(_randn(t.shape[0], 32)), w, out=t)


@pytest.mark.parametrize("write", [_rotate_in_place, _product_in_place])
def test_a_write_in_place_is_seen_by_autograd(write):
    # exp saves its result; once that is overwritten, backward must not use it
    x = _randn(6, 16).requires_grad_()
    y = x.exp()
    loss = y.sum()
    with torch.no_grad():
        write(y)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
    # what is not saved may be overwritten
    x.grad = None
    y = x * 2.0
    loss = y.sum()
    with torch.no_grad():
        write(y)
    loss.backward()
    assert (x.grad == 2.0).all()


@pytest.mark.parametrize("write", [_rotate_in_place, _product_in_place])
def test_versions_move_once_a_write(write):
    t = _randn(6, 16)
    for n in range(3):
        before = t._version
        write(t)
        assert t._version == before + 1
    # a refused call writes nothing
    before = t._version
    with pytest.raises(ValueError):
        kl.rope_axes(t.view(6, 2, 8), torch.zeros(5, 1, dtype=torch.int32, device="cuda"), (4,), out=t.view(6, 2, 8))
    assert t._version == before


@pytest.mark.parametrize("write", [_rotate_in_place, _product_in_place])
def test_inference_tensors_are_written(write):
    want = _randn(6, 16)
    write(want)
    with torch.inference_mode():
        t = _randn(6, 16)
        write(t)
        assert torch.equal(t, want)
    write(t)
