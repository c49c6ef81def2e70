"""The eight-bit projection path, plain fp64 definitions (TEST INFRASTRUCTURE
ONLY: imported by tests/, never by the library).

* FP8 encode: E4M3 codes with one power-of-two scale per block of 128 columns
  of a row, or per 128 x 128 tile: 2^e with e the least integer for which
  amax <= 448 * 2^e, clamped to [-127, 127], 0 for an all-zero block; codes are
  e4m3(x * 2^-e), nearest, ties to even.
* the product of two such operands, over their decoded values;
* rotary positions with several axes, and their inverse;
* LayerNorm and its gradients.
"""

import numpy as np

from .codecs import e4m3_decode, e4m3_encode


def block_exponents(x, block="row"):
    """Exponent e of each (row, block of 128 columns) of x; for "tile" the
    blocks of a 128-row group share theirs."""
    x = np.abs(np.asarray(x, np.float64))
    R, C = x.shape
    nb = -(-C // 128)
    amax = np.zeros((R, nb))
    for b in range(nb):
        amax[:, b] = x[:, b * 128:(b + 1) * 128].max(axis=1)
    if block == "tile":
        for r in range(0, R, 128):
            amax[r:r + 128] = amax[r:r + 128].max(axis=0)
    e = np.full(amax.shape, -127)
    for k in range(-127, 128):  # raised while the amax does not fit
        e = np.where(amax > 448.0 * 2.0 ** (e.astype(np.float64)), np.minimum(e + 1, 127), e)
    return np.where(amax == 0, 0, e)


def fp8_encode(x, block="row"):
    """(codes uint8 [R, C], e [R, ceil(C/128)])."""
    x = np.asarray(x, np.float64)
    e = block_exponents(x, block)
    s = np.repeat(2.0 ** -e.astype(np.float64), 128, axis=1)[:, :x.shape[1]]
    return e4m3_encode(x * s), e


def fp8_decode(codes, e):
    s = np.repeat(2.0 ** e.astype(np.float64), 128, axis=1)[:, :codes.shape[1]]
    return e4m3_decode(codes) * s


def scales_mma(e):
    """Scale bytes e + 127 in the product's layout: 512-byte atoms of 128 rows x
    4 blocks, byte (row%32)*16 + ((row/32)%4)*4 + block%4; the rest 0."""
    R, nb = e.shape
    ka = -(-nb // 4)
    out = np.zeros(-(-R // 128) * ka * 512, np.uint8)
    for b in range(nb):
        r = np.arange(R)
        out[((r // 128) * ka + b // 4) * 512 + (r % 32) * 16 + (r // 32 % 4) * 4 + b % 4] = e[:, b] + 127
    return out


def rope_axes(x, pos, sections, theta=10000.0, pairing="interleaved", ladder="axis", inverse=False):
    """x [..., tokens, heads, dim], pos [..., tokens, axes] -> rotated x.  Angles
    in extended precision."""
    x = np.asarray(x, np.float64)
    P = int(sum(sections))
    phi, j = [], 0
    for a, n in enumerate(sections):
        for u in range(n):
            ex = np.longdouble(u) / n if ladder == "axis" else np.longdouble(j) / P
            phi.append(np.asarray(pos)[..., a].astype(np.longdouble) * np.longdouble(theta) ** -ex)
            j += 1
    phi = np.stack(phi, -1)[..., None, :] * (-1 if inverse else 1)
    c, s = np.cos(phi).astype(np.float64), np.sin(phi).astype(np.float64)
    out = x.copy()
    i0, i1 = (np.arange(P), np.arange(P) + P) if pairing == "half" else (2 * np.arange(P), 2 * np.arange(P) + 1)
    out[..., i0] = x[..., i0] * c - x[..., i1] * s
    out[..., i1] = x[..., i0] * s + x[..., i1] * c
    return out


def _factor(gain, modulate, rows, cols):
    if gain is None:
        return np.ones((rows, cols))
    g = np.atleast_2d(np.asarray(gain, np.float64))
    return np.repeat(g + (1.0 if modulate else 0.0), rows // g.shape[0], axis=0)


def layer_norm(x, gain=None, bias=None, modulate=False, eps=1e-6):
    """(y, mean, rstd) of x [rows, cols]."""
    x = np.asarray(x, np.float64)
    mean = x.mean(axis=1)
    rstd = 1.0 / np.sqrt(((x - mean[:, None]) ** 2).mean(axis=1) + eps)
    y = (x - mean[:, None]) * rstd[:, None] * _factor(gain, modulate, *x.shape)
    if bias is not None:
        b = np.atleast_2d(np.asarray(bias, np.float64))
        y = y + np.repeat(b, x.shape[0] // b.shape[0], axis=0)
    return y, mean, rstd


def layer_norm_backward(dy, x, mean, rstd, gain=None, modulate=False, groups=1):
    """(dx, dgain, dbias) with the given row statistics."""
    dy, x = np.asarray(dy, np.float64), np.asarray(x, np.float64)
    mean, rstd = np.asarray(mean, np.float64)[:, None], np.asarray(rstd, np.float64)[:, None]
    xhat = (x - mean) * rstd
    h = dy * _factor(gain, modulate, *x.shape)
    dx = rstd * (h - h.mean(axis=1, keepdims=True) - xhat * (h * xhat).mean(axis=1, keepdims=True))
    shape = (groups, -1, x.shape[1])
    return dx, (dy * xhat).reshape(shape).sum(axis=1), dy.reshape(shape).sum(axis=1)
