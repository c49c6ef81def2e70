"""Pins of the eight-bit projection path's fp64 definitions: library codecs,
closed forms, brute force, torch's fp64 autograd and central differences."""

import math

import numpy as np
import pytest
import torch

from oracle import block, codecs, projection as P


def _rand(shape, seed, std=1.0):
    return np.random.RandomState(seed).randn(*shape).astype(np.float32).astype(np.float64) * std


@pytest.mark.parametrize("shape", [(1, 1), (3, 128), (5, 300), (130, 129)])
@pytest.mark.parametrize("kind", ["row", "tile"])
def test_block_exponent_is_the_least_that_fits(shape, kind):
    x = _rand(shape, 1) * 10.0 ** np.random.RandomState(2).randint(-6, 7, (shape[0], 1))
    e = P.block_exponents(x, kind)
    for r in range(shape[0]):
        for b in range(e.shape[1]):
            rows = slice(r, r + 1) if kind == "row" else slice(r // 128 * 128, r // 128 * 128 + 128)
            amax = np.abs(x[rows, b * 128:(b + 1) * 128]).max()
            assert amax <= 448 * 2.0 ** int(e[r, b]) and amax > 448 * 2.0 ** (int(e[r, b]) - 1)


def test_block_exponent_edges():
    x = np.array([[448.0], [448.0000001], [0.0], [2.0 ** -149], [3.4e38], [1.0], [1.75], [1.76]])
    assert P.block_exponents(x)[:, 0].tolist() == [0, 1, 0, -127, 120, -8, -8, -7]


def test_codes_match_the_library_codec_and_never_saturate():
    x = _rand((64, 512), 3)
    codes, e = P.fp8_encode(x)
    s = torch.from_numpy(np.repeat(2.0 ** -e, 128, axis=1))
    want = (torch.from_numpy(x) * s).float().to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    np.testing.assert_array_equal(codes, want)
    # half a step of E4M3 at each value, or of its least step 2^-9
    d = np.abs(P.fp8_decode(codes, e) - x)
    assert np.all(d <= np.maximum(np.abs(x) * 2.0 ** -4, np.repeat(2.0 ** e, 128, axis=1) * 2.0 ** -10))


def test_scale_layout_by_brute_force():
    e = np.random.RandomState(4).randint(-20, 20, (200, 6))
    m = P.scales_mma(e)
    assert m.size == 2 * 2 * 512
    seen = np.zeros(m.size, bool)
    for r in range(200):
        for b in range(6):
            atom = (r // 128) * 2 + b // 4
            at = atom * 512 + (r % 32) * 16 + (r % 128 // 32) * 4 + b % 4
            assert m[at] == e[r, b] + 127 and not seen[at]
            seen[at] = True
    assert np.all(m[~seen] == 0)


@pytest.mark.parametrize("pairing", ["interleaved", "half"])
@pytest.mark.parametrize("ladder", ["axis", "shared"])
def test_rope_is_a_rotation_and_its_inverse(pairing, ladder):
    x = _rand((7, 2, 22), 5)
    pos = np.random.RandomState(6).randint(0, 100, (7, 3))
    kw = dict(sections=(3, 4, 2), pairing=pairing, ladder=ladder)
    y = P.rope_axes(x, pos, **kw)
    np.testing.assert_allclose((y ** 2).sum(-1), (x ** 2).sum(-1), rtol=1e-12)
    np.testing.assert_array_equal(y[..., 18:], x[..., 18:])
    np.testing.assert_allclose(P.rope_axes(y, pos, inverse=True, **kw), x, atol=1e-12)
    np.testing.assert_array_equal(P.rope_axes(x, pos * 0, **kw), x)
    # the gradient of sum(y * g) with respect to x is the inverse rotation of g
    g, d = _rand(x.shape, 7), _rand(x.shape, 8)
    lhs = (P.rope_axes(d, pos, **kw) * g).sum()
    assert abs(lhs - (d * P.rope_axes(g, pos, inverse=True, **kw)).sum()) <= 1e-10


def test_rope_matches_the_blocks_angles_on_image_tokens():
    lay = block.TokenLayout(0, 4, 5, 1)
    f, r, c = np.meshgrid(range(2), range(4), range(5), indexing="ij")
    pos = np.stack([f, r, c], -1).reshape(-1, 3)
    x = _rand((40, 2, 128), 9)
    np.testing.assert_allclose(P.rope_axes(x, pos, (16, 24, 24)), block.apply_rope(x, block.rope_angles(lay)),
                               atol=1e-12)


def test_rope_quarter_turn_closed_form():
    # theta^(-1/1 * 0) = 1: one pair, position pi/2 turns (1, 0) into (0, 1)
    y = P.rope_axes(np.array([[[1.0, 0.0]]]), np.array([[math.pi / 2]]), (1,))
    np.testing.assert_allclose(y[0, 0], [0.0, 1.0], atol=1e-15)


@pytest.mark.parametrize("modulate", [False, True])
@pytest.mark.parametrize("groups", [1, 3])
def test_layer_norm_matches_torch_autograd(modulate, groups):
    R, C = 12, 37
    x = torch.from_numpy(_rand((R, C), 10) + 3).requires_grad_()
    g = torch.from_numpy(_rand((groups, C), 11)).requires_grad_()
    b = torch.from_numpy(_rand((groups, C), 12)).requires_grad_()
    dy = torch.from_numpy(_rand((R, C), 13))
    f = g.repeat_interleave(R // groups, 0) + (1 if modulate else 0)
    y = torch.nn.functional.layer_norm(x, (C,), eps=1e-6) * f + b.repeat_interleave(R // groups, 0)
    y.backward(dy)
    got, mean, rstd = P.layer_norm(x.detach().numpy(), g.detach().numpy(), b.detach().numpy(), modulate)
    np.testing.assert_allclose(got, y.detach().numpy(), atol=1e-11)
    dx, dg, db = P.layer_norm_backward(dy.numpy(), x.detach().numpy(), mean, rstd, g.detach().numpy(), modulate, groups)
    np.testing.assert_allclose(dx, x.grad.numpy(), atol=1e-11)
    np.testing.assert_allclose(dg, g.grad.numpy(), atol=1e-11)
    np.testing.assert_allclose(db, b.grad.numpy(), atol=1e-11)


def test_layer_norm_gradient_against_differences():
    x, dy, g = _rand((2, 9), 14), _rand((2, 9), 15), _rand((9,), 16)
    _, mean, rstd = P.layer_norm(x, g)
    dx, _, _ = P.layer_norm_backward(dy, x, mean, rstd, g)
    h = 1e-6
    for r in range(2):
        for c in range(9):
            d = np.zeros_like(x)
            d[r, c] = h
            diff = ((P.layer_norm(x + d, g)[0] - P.layer_norm(x - d, g)[0]) * dy).sum() / (2 * h)
            assert abs(diff - dx[r, c]) <= 1e-6 * (1 + abs(diff))


def test_decoded_product_equals_integers_exactly():
    # whole numbers up to 16 are E4M3 values at any power of two: the product is the integers'
    rs = np.random.RandomState(17)
    a, w = rs.randint(-16, 17, (5, 200)).astype(np.float64), rs.randint(-16, 17, (7, 200)).astype(np.float64)
    da, dw = P.fp8_decode(*P.fp8_encode(a * 2.0 ** 20)), P.fp8_decode(*P.fp8_encode(w * 2.0 ** -20, "tile"))
    np.testing.assert_array_equal(da @ dw.T, a @ w.T)
    assert codecs.e4m3_round(16.0) == 16.0
