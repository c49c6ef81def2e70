"""kl_layer_norm_forward / backward against the fp64 definitions."""

import numpy as np
import pytest
import torch

import diffusion_transformer_image_nvfp4_b200 as kl
from oracle import projection as P

pytestmark = pytest.mark.gpu

HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
LEAST = {torch.bfloat16: 0.0, torch.float16: 2.0 ** -25, torch.float32: 0.0}
# a sum over a row passes through at most 32 additions in a thread, 5 in its
# warp and 32 over the warps; with the roundings of the terms, 96 units of 2^-24
# of the sum of magnitudes (rows of up to 32 * 1024 columns)
ROW = 96 * 2.0 ** -24
U = 2.0 ** -24


def _np(t):
    return None if t is None else t.detach().cpu().double().numpy()


def _randn(shape, seed, dtype, scale=1.0, off=0.0):
    return (torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * scale + off).to(dtype).cuda()


def _params(kind, groups, C, dtype, seed):
    if kind == "none":
        return None, None
    base = 0.0 if kind == "modulate" else 1.0
    return _randn((groups, C), seed, dtype, 0.3, base), _randn((groups, C), seed + 1, dtype, 0.3)


def _rep(g, rows):
    return np.repeat(g, rows // g.shape[0], axis=0)


def _check_forward(y, mean, rstd, x, gain, bias, modulate):
    X = _np(x.reshape(-1, x.shape[-1]))
    ref, m, r = P.layer_norm(X, _np(gain), _np(bias), modulate)
    am = np.abs(X).mean(1)
    assert np.all(np.abs(_np(mean) - m) <= ROW * am + U * np.abs(m))
    # the mean's error e adds e^2 to the variance; the variance's own sum is
    # off by ROW of itself, and rstd by half of that and two roundings
    e = ROW * am + U * np.abs(m)
    rtol = 0.5 * (ROW + e * e * r * r) + 4 * U
    assert np.all(np.abs(_np(rstd) - r) <= rtol * r)
    f = np.abs(P._factor(_np(gain), modulate, *X.shape))
    xh = np.abs(X - m[:, None]) * r[:, None]
    tol = f * (xh * (rtol[:, None] + 4 * U) + (e * r)[:, None]) + 2 * U * np.abs(ref)
    if bias is not None:
        tol = tol + 2 * U * np.abs(_rep(_np(bias), len(X)))
    tol = tol * (1 + HALF_STEP[x.dtype]) + HALF_STEP[x.dtype] * np.abs(ref) + LEAST[x.dtype]
    d = np.abs(_np(y).reshape(X.shape) - ref)
    assert np.all(d <= tol), (d - tol).max()


def _check_backward(got, dy, x, mean, rstd, gain, modulate, groups):
    dx, dg, db = got
    X, D = _np(x.reshape(-1, x.shape[-1])), _np(dy.reshape(-1, x.shape[-1]))
    R, C = X.shape
    ref, rg, rb = P.layer_norm_backward(D, X, _np(mean), _np(rstd), _np(gain), modulate, groups)
    r = _np(rstd)[:, None]
    xh = np.abs(X - _np(mean)[:, None]) * r
    h = np.abs(D * P._factor(_np(gain), modulate, R, C))
    # row sums as above; h and xhat carry two roundings each, the last
    # expression four
    m0 = (ROW + 2 * U) * h.mean(1, keepdims=True)
    m1 = (ROW + 4 * U) * (h * xh).mean(1, keepdims=True)
    tol = r * (m0 + xh * m1 + 6 * U * (h + h.mean(1, keepdims=True) + xh * (h * xh).mean(1, keepdims=True)))
    tol = tol * (1 + HALF_STEP[x.dtype]) + HALF_STEP[x.dtype] * np.abs(ref) + LEAST[x.dtype]
    d = np.abs(_np(dx).reshape(X.shape) - ref)
    assert np.all(d <= tol), (d - tol).max()
    if dg is None:
        return
    # a column's sum: the rows of one thread, then thread rows and partials
    depth = min(R, 512) + 64
    shape = (groups, -1, C)
    assert np.all(np.abs(_np(dg) - rg) <= depth * U * np.abs(D * xh).reshape(shape).sum(1) + 1e-37)
    assert np.all(np.abs(_np(db) - rb) <= depth * U * np.abs(D).reshape(shape).sum(1) + 1e-37)


# widths of single elements and of vectors, one to many threads a row, one and
# two vectors a thread, the widest register rows and the re-reading kernels
WIDTHS = [1, 2, 7, 8, 31, 64, 128, 200, 257, 1000, 1155, 2049, 3072, 4096, 4100, 8192, 8200, 9001, 33000]


@pytest.mark.parametrize("C", WIDTHS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_forward_and_backward(C, dtype):
    for R, groups, kind, pt in ((1, 1, "none", dtype), (6, 3, "modulate", dtype), (37, 1, "gain", torch.float32)):
        x = _randn((R, C), R + C, dtype, 1.5, 0.5)
        gain, bias = _params(kind, groups, C, pt, C)
        mod = kind == "modulate"
        y, mean, rstd = kl.layer_norm_forward(x, gain, bias, modulate=mod)
        _check_forward(y, mean, rstd, x, gain, bias, mod)
        dy = _randn((R, C), R + C + 1, dtype)
        got = kl.layer_norm_backward(dy, x, mean, rstd, gain, modulate=mod, groups=groups)
        _check_backward(got, dy, x, mean, rstd, gain, mod, groups)
        dx, dg, db = kl.layer_norm_backward(dy, x, mean, rstd, gain, modulate=mod, groups=groups, param_grads=False)
        assert dg is None and db is None and torch.equal(dx, got[0])
    assert kl.device_status() == "KL_OK"


@pytest.mark.parametrize("R,C,groups", [(5000, 128, 2), (4099, 384, 1), (1001, 1155, 7), (600, 3072, 600),
                                        (3000, 24, 3), (700, 9001, 1)])
def test_many_rows_and_groups(R, C, groups):
    for dtype in (torch.bfloat16, torch.float32):
        x, dy = _randn((R, C), 1, dtype, 2.0, 1.0), _randn((R, C), 2, dtype)
        gain, bias = _params("modulate", groups, C, torch.bfloat16, 3)
        y, mean, rstd = kl.layer_norm_forward(x, gain, bias, modulate=True)
        _check_forward(y, mean, rstd, x, gain, bias, True)
        got = kl.layer_norm_backward(dy, x, mean, rstd, gain, modulate=True)
        _check_backward(got, dy, x, mean, rstd, gain, True, groups)
        again = kl.layer_norm_backward(dy, x, mean, rstd, gain, modulate=True)
        assert all(torch.equal(a, b) for a, b in zip(got, again))


@pytest.mark.parametrize("R,C,groups", [(1205, 3072, 1), (2402, 1536, 2), (5001, 512, 1), (1210, 8192, 2),
                                        (9000, 256, 3), (1300, 4096, 1)])
def test_staged_tiles_of_rows(R, C, groups):
    # rows enough for every SM: tiles of rows in shared memory, the last of a group ragged
    for dtype in (torch.bfloat16, torch.float16, torch.float32):
        x, dy = _randn((R, C + 16), 1, dtype, 2.0, 1.0)[:, 16:], _randn((R, C), 2, dtype)
        gain, bias = _params("gain", groups, C, torch.float32, 3)
        y, mean, rstd = kl.layer_norm_forward(x, gain, bias)
        _check_forward(y, mean, rstd, x, gain, bias, False)
        got = kl.layer_norm_backward(dy, x, mean, rstd, gain)
        _check_backward(got, dy, x, mean, rstd, gain, False, groups)
        again = kl.layer_norm_backward(dy, x, mean, rstd, gain)
        assert all(torch.equal(a, b) for a, b in zip(got, again))
        dx = kl.layer_norm_backward(dy, x, mean, rstd, gain, param_grads=False)[0]
        assert torch.equal(dx, got[0])
    assert kl.device_status() == "KL_OK"


@pytest.mark.parametrize("R,C,groups", [(1205, 258, 1), (2402, 1022, 2), (1501, 1026, 1), (1210, 4094, 2), (900, 2934, 3),
                                        (700, 6142, 1), (3000, 34, 2)])
def test_many_rows_of_even_width(R, C, groups):
    # two elements at a time where x, dy and the results start on them, else one
    for dtype in (torch.bfloat16, torch.float16, torch.float32):
        wide = _randn((R, C + 3), 1, dtype, 2.0, 1.0)
        gain, bias = _params("gain", groups, C, torch.float32, 3)
        for x in (wide[:, 2:C + 2].contiguous(), wide[:, 1:C + 1]):
            y, mean, rstd = kl.layer_norm_forward(x, gain, bias)
            _check_forward(y, mean, rstd, x, gain, bias, False)
            dy = _randn((R, C), 2, dtype)
            got = kl.layer_norm_backward(dy, x, mean, rstd, gain)
            _check_backward(got, dy, x, mean, rstd, gain, False, groups)


@pytest.mark.parametrize("R,C,groups", [(1205, 257, 1), (2402, 1023, 2), (1501, 1025, 1), (1210, 4095, 2), (900, 2047, 3),
                                        (700, 6143, 1), (3000, 33, 2)])
def test_many_rows_of_odd_width(R, C, groups):
    for dtype in (torch.bfloat16, torch.float16, torch.float32):
        x, dy = _randn((R, C), 1, dtype, 2.0, 1.0), _randn((R, C + 1), 2, dtype)[:, 1:]
        gain, bias = _params("modulate", groups, C, dtype, 3)
        y, mean, rstd = kl.layer_norm_forward(x, gain, bias, modulate=True)
        _check_forward(y, mean, rstd, x, gain, bias, True)
        got = kl.layer_norm_backward(dy, x, mean, rstd, gain, modulate=True)
        _check_backward(got, dy, x, mean, rstd, gain, True, groups)
        assert torch.equal(kl.layer_norm_backward(dy, x, mean, rstd, gain, modulate=True, param_grads=False)[0], got[0])


@pytest.mark.parametrize("R,C,groups", [(400, 64, 1), (401, 64, 1), (399, 3072, 1), (800, 1155, 2), (1600, 2048, 4),
                                        (1024, 1024, 512), (2, 40, 2)])
def test_one_and_two_launches(R, C, groups):
    # on both sides of where the parameters' sums take a launch of their own
    for dtype in (torch.bfloat16, torch.float32):
        x, dy = _randn((R, C), 1, dtype, 2.0, 1.0), _randn((R, C), 2, dtype)
        gain, bias = _params("gain", groups, C, dtype, 3)
        _, mean, rstd = kl.layer_norm_forward(x, gain, bias)
        got = kl.layer_norm_backward(dy, x, mean, rstd, gain)
        _check_backward(got, dy, x, mean, rstd, gain, False, groups)
        assert all(torch.equal(a, b) for a, b in zip(got, kl.layer_norm_backward(dy, x, mean, rstd, gain)))


def test_strides_batches_and_alignment():
    big, dbig = _randn((30, 1000), 4, torch.bfloat16, 2.0), _randn((30, 1000), 5, torch.bfloat16)
    for cut in (lambda t: t[:, 8:520], lambda t: t[:, 3:300], lambda t: t.view(6, 5, 1000)[:, 2, :640],
                lambda t: t.view(2, 15, 1000)[..., 16:48]):
        x, dy = cut(big), cut(dbig)
        C = x.shape[-1]
        gain, bias = _randn((C + 1,), 6, torch.float32)[1:].clone(), _randn((C,), 7, torch.float32)
        y, mean, rstd = kl.layer_norm_forward(x, gain, bias)
        assert y.shape == x.shape
        _check_forward(y, mean, rstd, x, gain[None], bias[None], False)
        got = kl.layer_norm_backward(dy, x, mean, rstd, gain)
        _check_backward(got, dy, x, mean, rstd, gain[None], False, 1)
        # parameters that do not start on 16 bytes
        off = torch.empty(C + 1, device="cuda")
        off[1:] = gain
        assert torch.equal(kl.layer_norm_forward(x, off[1:], bias)[0], y)
        # gain alone, bias alone
        _check_forward(*kl.layer_norm_forward(x, gain), x, gain[None], None, False)
        _check_forward(*kl.layer_norm_forward(x, None, bias), x, None, bias[None], False)


def test_offset_rows_constant_rows_and_large_values():
    # a common offset 4096 times the spread; a constant row; values near the type's top
    x = _randn((4, 512), 8, torch.float32)
    x[0] += 4096.0
    x[1] = 3.0
    x[2] *= 1e15
    y, mean, rstd = kl.layer_norm_forward(x)
    _check_forward(y, mean, rstd, x, None, None, False)
    assert (y[1] == 0).all() and torch.isfinite(y).all()
    dy = _randn((4, 512), 9, torch.float32)
    got = kl.layer_norm_backward(dy, x, mean, rstd)
    _check_backward(got, dy, x, mean, rstd, None, False, 1)


def test_nonfinite_rows_stay_alone():
    x = _randn((9, 300), 10, torch.bfloat16)
    clean = kl.layer_norm_forward(x)[0]
    x[4, 17], x[7, 0] = float("nan"), float("inf")
    y, mean, rstd = kl.layer_norm_forward(x)
    assert torch.isnan(y[4]).all() and torch.isnan(y[7]).all()
    rest = [0, 1, 2, 3, 5, 6, 8]
    assert torch.equal(y[rest], clean[rest])
    dx = kl.layer_norm_backward(torch.ones_like(x), x, mean, rstd, param_grads=False)[0]
    assert torch.isfinite(dx[rest]).all() and torch.isnan(dx[4]).all()


def test_gradients_against_differences():
    x, dy = _randn((3, 40), 11, torch.float32), _randn((3, 40), 12, torch.float32)
    gain, bias = _params("modulate", 1, 40, torch.float32, 13)
    _, mean, rstd = kl.layer_norm_forward(x, gain, bias, modulate=True)
    dx, dg, db = kl.layer_norm_backward(dy, x, mean, rstd, gain, modulate=True)
    f = lambda X, G, B: (P.layer_norm(X, G, B, True)[0] * _np(dy)).sum()
    X, G, B, h = _np(x), _np(gain), _np(bias), 1e-5
    for at in ((0, 0), (1, 17), (2, 39)):
        d = np.zeros_like(X)
        d[at] = h
        assert abs((f(X + d, G, B) - f(X - d, G, B)) / (2 * h) - float(dx[at])) <= 1e-5
    for c in (0, 20, 39):
        d = np.zeros_like(G)
        d[0, c] = h
        assert abs((f(X, G + d, B) - f(X, G - d, B)) / (2 * h) - float(dg[0, c])) <= 2e-5
        assert abs((f(X, G, B + d) - f(X, G, B - d)) / (2 * h) - float(db[0, c])) <= 2e-5


def test_two_streams_at_once_and_two_graphs():
    # every call has its own scratch: calls that overlap do not disturb each other
    xs = [_randn((900, 1024), 14 + k, torch.bfloat16) for k in range(2)]
    st = [kl.layer_norm_forward(x) for x in xs]
    want = [kl.layer_norm_backward(x, x, m, r) for x, (_, m, r) in zip(xs, st)]
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(8):
        for k, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[k].append(kl.layer_norm_backward(xs[k], xs[k], st[k][1], st[k][2]))
    torch.cuda.synchronize()
    for k in range(2):
        for g in got[k]:
            assert all(torch.equal(a, b) for a, b in zip(g, want[k]))
    graphs = []
    for k in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = kl.layer_norm_backward(xs[k], xs[k], st[k][1], st[k][2])
        graphs.append((g, out))
    for k in (0, 1, 0, 1):
        with torch.cuda.stream(streams[k]):
            graphs[k][0].replay()
    torch.cuda.synchronize()
    for k in range(2):
        assert all(torch.equal(a, b) for a, b in zip(graphs[k][1], want[k]))


def test_matches_the_blocks_own_layer_norm():
    # the block's m = bf16(LN(x)(1 + scale) + shift) to one bf16 step
    x, sc, sh = (_randn(s, 20 + k, torch.bfloat16) for k, s in enumerate(((300, 512), (512,), (512,))))
    m, _ = kl.ln_modulate_bf16(x, sh, sc)
    y = kl.layer_norm_forward(x, sc, sh, modulate=True)[0]
    d = (m.float() - y.float()).abs()
    assert (d <= m.float().abs() * 2.0 ** -7 + 1e-6).all() and (d == 0).float().mean() > 0.99


def test_refusals():
    x = _randn((6, 32), 21, torch.float32)
    y, mean, rstd = kl.layer_norm_forward(x)
    g = torch.ones(32, device="cuda")
    for call in (lambda: kl.layer_norm_forward(x, g[:31]), lambda: kl.layer_norm_forward(x, g.double()),
                 lambda: kl.layer_norm_forward(x, g.expand(4, 32).contiguous()),
                 lambda: kl.layer_norm_forward(x, g, g.half()), lambda: kl.layer_norm_forward(x, g, g.expand(2, 32).contiguous()),
                 lambda: kl.layer_norm_forward(x.t()), lambda: kl.layer_norm_forward(x[:0]),
                 lambda: kl.layer_norm_backward(x[:5], x, mean, rstd), lambda: kl.layer_norm_backward(x.half(), x, mean, rstd),
                 lambda: kl.layer_norm_backward(x, x, mean[:5], rstd), lambda: kl.layer_norm_backward(x, x, mean.double(), rstd),
                 lambda: kl.layer_norm_backward(x, x, mean, rstd, groups=4),
                 lambda: kl.layer_norm_backward(x[:1].expand(6, 32), x, mean, rstd)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(kl.KLError, match="INVALID_ARG"):
        kl.layer_norm_forward(x, eps=-1.0)
