"""The projection path's calls beside torch's autograd: what they write in place
is seen by it, and no tensor that requires a gradient is taken while it records."""

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


def _calls():
    """(call, its tensors): every place that takes a floating tensor."""
    x, dy, g, b = _randn(6, 16), _randn(6, 16).flip(0).contiguous(), _randn(16), _randn(16)
    _, mean, rstd = kl.layer_norm_forward(x)
    heads, pos = _randn(6, 2, 8), torch.arange(6.0, device="cuda")[:, None]
    w = kl.quantize_fp8_block(_randn(16, 32))
    a = kl.quantize_fp8_block(_randn(6, 32))
    return {
        "encode": (lambda x: kl.quantize_fp8_block(x).codes, [x]),
        "product": (lambda out: kl.gemm_fp8_block(a, w, out=out), [_randn(6, 16)]),
        "rotary": (lambda x, pos, out: kl.rope_axes(x, pos, (4,), out=out), [heads, pos, _randn(6, 2, 8)]),
        "layer norm": (lambda x, g, b: kl.layer_norm_forward(x, g, b), [x, g, b]),
        "layer norm backward": (lambda *t: kl.layer_norm_backward(*t), [dy, x, mean, rstd, g]),
    }


def test_tensors_that_require_a_gradient_are_refused_in_every_place():
    for name, (call, tensors) in _calls().items():
        want = call(*tensors)
        want = [t.clone() for t in (want if isinstance(want, tuple) else (want,))]
        for k in range(len(tensors)):
            with_leaf = [t.clone().requires_grad_() if i == k else t for i, t in enumerate(tensors)]
            with pytest.raises(ValueError, match="requires a gradient"):
                call(*with_leaf)
            with torch.no_grad():
                got = call(*with_leaf)
            got = got if isinstance(got, tuple) else (got,)
            assert all(torch.equal(a, b) for a, b in zip(got, want)), name


class _LayerNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, gain, bias):
        y, mean, rstd = kl.layer_norm_forward(x, gain, bias)
        ctx.save_for_backward(x, mean, rstd, gain)
        return y

    @staticmethod
    def backward(ctx, dy):
        dx, dgain, dbias = kl.layer_norm_backward(dy, *ctx.saved_tensors)
        return dx, dgain[0], dbias[0]


def test_the_two_forms_make_an_autograd_function():
    leaves = [t.requires_grad_() for t in (_randn(6, 16), _randn(16), _randn(1, 16)[0])]
    dy = _randn(6, 16)
    got = torch.autograd.grad(_LayerNorm.apply(*leaves), leaves, dy)
    x, g, b = (t.detach().double().requires_grad_() for t in leaves)
    y = torch.nn.functional.layer_norm(x, (16,), g, b, eps=1e-6)
    for a, r in zip(got, torch.autograd.grad(y, (x, g, b), dy.double())):
        # at most 16 terms a sum: 64 units of 2^-24 of the largest magnitude met, rstd * |xhat| * max|h xhat|
        # <= 1.4 * 3.6 * 26 < 132 for these inputs
        assert (a.double() - r).abs().max() <= 64 * 2.0 ** -24 * 132
    # a second derivative is not provided, and says so
    out = _LayerNorm.apply(*leaves)
    with pytest.raises(ValueError, match="requires a gradient"):
        torch.autograd.grad(out, leaves, dy.requires_grad_(), create_graph=True)
