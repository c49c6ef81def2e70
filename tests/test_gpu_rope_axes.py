"""kl_rope_axes against the fp64 definition."""

import numpy as np
import pytest
import torch

import diffusion_transformer_image_nvfp4_b200 as kl
from oracle import projection as P

pytestmark = pytest.mark.gpu

HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}


def _np(t):
    return t.detach().cpu().double().numpy()


def _randn(shape, seed, dtype):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


def _check(got, x, pos, sections, angle_err=0.0, **kw):
    """The angle is rounded to fp32 once within half a turn (2^-24 * pi), cos
    and sin are off by two units (2^-22), two products and their sum round in
    fp32: 8e-7 of each of the pair's values, then the output's half step (its
    least step 2^-25 for fp16)."""
    ref = P.rope_axes(_np(x), pos.cpu().numpy(), sections, **kw)
    n = sum(sections)
    xa = np.abs(_np(x))
    mag = np.zeros_like(xa)
    i0, i1 = (np.arange(n), np.arange(n) + n) if kw.get("pairing") == "half" else (2 * np.arange(n), 2 * np.arange(n) + 1)
    mag[..., i0] = mag[..., i1] = xa[..., i0] + xa[..., i1]
    tol = (8e-7 + angle_err) * mag * 1.01 + HALF_STEP[x.dtype] * np.abs(ref) + (2.0 ** -25 if x.dtype == torch.float16 else 0)
    d = np.abs(_np(got) - ref)
    assert np.all(d <= tol), (d - tol).max()
    np.testing.assert_array_equal(_np(got)[..., 2 * n:], _np(x)[..., 2 * n:])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("pairing", ["interleaved", "half"])
@pytest.mark.parametrize("ladder", ["axis", "shared"])
@pytest.mark.parametrize("T,H,dim,sections", [(1, 1, 2, (1,)), (5, 3, 128, (16, 24, 24)), (40, 2, 96, (8, 16, 16)),
                                              (7, 5, 23, (3, 4)), (33, 24, 64, (4, 4, 4, 4)), (9, 1, 512, (256,)),
                                              (6, 2, 20, (0, 6)), (3, 40, 100, (10, 30))])
def test_matches_definition(T, H, dim, sections, pairing, ladder, dtype):
    x = _randn((T, H, dim), T + dim, dtype)
    g = torch.Generator().manual_seed(dim)
    for pt in (torch.int32, torch.int64, torch.float32):
        pos = torch.randint(0, 200, (T, len(sections)), generator=g)
        pos = (pos.float() * 0.37 if pt == torch.float32 else pos.to(pt)).cuda()
        kw = dict(pairing=pairing, ladder=ladder)
        y = kl.rope_axes(x, pos, sections, **kw)
        _check(y, x, pos, sections, **kw)
        _check(kl.rope_axes(x, pos, sections, inverse=True, **kw), x, pos, sections, inverse=True, **kw)


def test_batches_strides_in_place_and_shared_positions():
    T, H = 37, 6
    buf = _randn((2, T, 3 * H, 128), 1, torch.bfloat16)
    pos = torch.randint(0, 64, (2, T, 3), generator=torch.Generator().manual_seed(2)).cuda()
    x = buf[:, :, :2 * H]
    keep, v = x.clone(), buf[:, :, 2 * H:].clone()
    y = kl.rope_axes(x, pos, (16, 24, 24))
    _check(y, keep, pos, (16, 24, 24))
    assert torch.equal(x, keep)
    out = torch.zeros(2, 2 * H, T, 128, dtype=torch.bfloat16, device="cuda").transpose(1, 2)
    assert torch.equal(kl.rope_axes(x, pos, (16, 24, 24), out=out), y)
    shared = kl.rope_axes(x, pos[0], (16, 24, 24))
    assert torch.equal(shared[0], y[0])
    _check(shared, keep, pos[:1].expand(2, T, 3), (16, 24, 24))
    assert kl.rope_axes(x, pos, (16, 24, 24), out=x) is x
    assert torch.equal(x, y) and torch.equal(buf[:, :, 2 * H:], v)
    odd = _randn((T, 4, 131), 3, torch.float16)[:, 1:3, 1:100]  # single elements
    for pairing in ("interleaved", "half"):
        _check(kl.rope_axes(odd, pos[0], (16, 24, 8), pairing=pairing), odd, pos[:1, :, :][0], (16, 24, 8),
               pairing=pairing)


@pytest.mark.parametrize("B,T,H,dim,sections", [(1, 2000, 3, 128, (16, 24, 24)), (3, 700, 40, 64, (5, 11)), (2, 5000, 1, 8, (2, 1)),
                                                (1, 2, 300, 128, (64,)), (5, 1, 7, 510, (255,)), (300, 3, 2, 16, (8,))])
def test_many_tokens_heads_and_batches(B, T, H, dim, sections):
    # several chunks a CTA, heads split over CTAs, chunks that end inside a batch
    for dtype in (torch.bfloat16, torch.float32):
        big = _randn((B, T, H + 1, dim + 8), 1, dtype)
        x = big[:, :, :H, :dim]
        pos = torch.randint(0, 500, (B, T, len(sections)), generator=torch.Generator().manual_seed(T)).int().cuda()
        for pairing in ("interleaved", "half"):
            y = kl.rope_axes(x, pos, sections, pairing=pairing)
            _check(y, x, pos, sections, pairing=pairing)
            out = torch.full_like(big, 3.0)
            kl.rope_axes(x, pos, sections, pairing=pairing, out=out[:, :, :H, :dim])
            assert torch.equal(out[:, :, :H, :dim], y)
            assert (out[:, :, H:] == 3).all() and (out[..., dim:] == 3).all()


@pytest.mark.parametrize("pt", [torch.int32, torch.int64, torch.float32])
def test_far_positions(pt):
    # one fp64 product of a rounded frequency: 3 * 2^-53 of the angle
    far = [0, 1, 65537, 10 ** 6 + 3, 2 ** 24 - 1, 2 ** 31 - 1]
    pos = torch.tensor(far, dtype=torch.float64).to(pt)[:, None].cuda()
    if pt == torch.int64:
        pos[-1] = 2 ** 40 + 1
    x = _randn((len(far), 3, 64), 4, torch.float32)
    err = 3 * 2.0 ** -53 * float(pos.max())
    _check(kl.rope_axes(x, pos, (32,)), x, pos, (32,), angle_err=err)
    neg = -pos
    _check(kl.rope_axes(x, neg, (32,)), x, neg, (32,), angle_err=err)


def test_nonfinite_values_stay_in_their_pair():
    x = _randn((4, 2, 32), 5, torch.bfloat16)
    x[1, 0, 4], x[2, 1, 30], x[3, 0, 31] = float("nan"), float("inf"), float("-inf")
    pos = torch.arange(4, dtype=torch.int32, device="cuda")[:, None] + 1
    y = kl.rope_axes(x, pos, (12,))  # dims 24.. are copied
    bad = ~torch.isfinite(y)
    assert bad.sum() == 4 and bad[1, 0, 4] and bad[1, 0, 5]
    assert torch.equal(y[..., 24:], x[..., 24:])


def test_same_angles_as_the_fused_table():
    # the QKV epilogue's table for image tokens, applied by hand
    lay = (0, 8, 6, 1)
    f, r, c = torch.meshgrid(torch.arange(2), torch.arange(8), torch.arange(6), indexing="ij")
    pos = torch.stack([f, r, c], -1).reshape(-1, 3).int().cuda()
    T = pos.shape[0]
    cs = kl.rope_table(*lay).permute(1, 0, 2, 3).reshape(T, 1, 64, 2)
    x = _randn((T, 3, 128), 6, torch.float32)
    a, b = x[..., 0::2], x[..., 1::2]
    want = torch.stack([a * cs[..., 0] - b * cs[..., 1], a * cs[..., 1] + b * cs[..., 0]], -1).flatten(-2)
    assert (kl.rope_axes(x, pos, (16, 24, 24)) - want).abs().max() <= 2e-6 * x.abs().max()


def test_gradient_against_differences():
    x, g = _randn((5, 2, 24), 7, torch.float32), _randn((5, 2, 24), 8, torch.float32)
    pos = torch.rand(5, 2, generator=torch.Generator().manual_seed(9)).cuda() * 50
    kw = dict(pairing="half", ladder="shared")
    grad = kl.rope_axes(g, pos, (5, 6), inverse=True, **kw)
    # the map is linear: a step of 1 has no error but rounding
    for at in ((0, 0, 0), (3, 1, 10), (4, 0, 13), (2, 1, 23)):
        d = torch.zeros_like(x)
        d[at] = 1.0
        diff = ((kl.rope_axes(x + d, pos, (5, 6), **kw) - kl.rope_axes(x, pos, (5, 6), **kw)) * g).double().sum()
        assert abs(float(diff) - float(grad[at])) <= 1e-5


def test_graph_and_side_stream():
    x, pos = _randn((6, 4, 64), 10, torch.bfloat16), torch.arange(6, device="cuda")[:, None]
    want = kl.rope_axes(x, pos, (32,))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = kl.rope_axes(x, pos, (32,))
    side.synchronize()
    assert torch.equal(got, want)
    buf, p = x.clone(), pos.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = kl.rope_axes(buf, p, (32,))
    buf.copy_(x * 2)
    p.copy_(pos + 100)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, kl.rope_axes(x * 2, pos + 100, (32,)))


def test_refusals():
    x, pos = _randn((4, 2, 32), 11, torch.float32), torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    for bad in (dict(pairing="pairs"), dict(ladder="one"), dict(out=torch.empty(4, 2, 31, device="cuda")),
                dict(out=x.half()), dict(out=torch.empty(4, 1, 32, device="cuda").expand(4, 2, 32))):
        with pytest.raises(ValueError):
            kl.rope_axes(x, pos, (8, 8), **bad)
    for p in (pos[:3], pos.double(), pos.cpu(), pos[:, :1]):
        with pytest.raises(ValueError):
            kl.rope_axes(x, p, (8, 8))
    with pytest.raises(kl.KLError, match="UNSUPPORTED_SHAPE"):
        kl.rope_axes(x, pos, (8, 9))
    with pytest.raises(kl.KLError, match="INVALID_ARG"):
        kl.rope_axes(x, pos, (8, 8), theta=0.5)
    with pytest.raises(ValueError):
        kl.rope_axes(x.transpose(1, 2), pos, (1, 0))
