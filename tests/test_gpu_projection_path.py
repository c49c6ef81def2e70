"""The eight-bit projection path end to end, as a layer uses it: LayerNorm with
modulation, encode, QKV product, rotary positions on q and k in place, joint
attention; and the same layer's backward pass up to the attention."""

import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import diffusion_transformer_image_nvfp4_b200 as kl
from oracle import block
from oracle import projection as P
from tests.helpers import rel_l2

pytestmark = pytest.mark.gpu

SECTIONS = (16, 24, 24)


def _np(t):
    return t.detach().cpu().double().numpy()


def _inputs(T, H, seed):
    g = torch.Generator().manual_seed(seed)
    D = H * 128
    x = (torch.randn(T, D, generator=g) * torch.exp(0.5 * torch.randn(T, 1, generator=g)) + 0.2).bfloat16().cuda()
    w = (torch.randn(3 * D, D, generator=g) / D ** 0.5).bfloat16().cuda()
    scale, shift = ((0.2 * torch.randn(1, D, generator=g)).bfloat16().cuda() for _ in range(2))
    pos = torch.stack([torch.zeros(T), torch.arange(T) // 16, torch.arange(T) % 16], 1).int().cuda()
    return x, w, scale, shift, pos


def _layer(x, W, scale, shift, pos, H):
    T, D = x.shape
    y, mean, rstd = kl.layer_norm_forward(x, scale, shift, modulate=True)
    qkv = kl.gemm_fp8_block(kl.quantize_fp8_block(y), W)
    before = qkv.clone()
    qk = qkv.view(T, 3 * H, 128)[:, :2 * H]
    kl.rope_axes(qk, pos, SECTIONS, out=qk)
    att = kl.joint_attention(qkv, qkv[:, D:], qkv[:, 2 * D:], T, H, 3 * D, "bf16")
    return y, mean, rstd, before, qkv, att


def _encode_error(x, e):
    """Most by which a value and its decoded code differ: half an E4M3 step,
    2^-4 of it, or half the least step, 2^-10, times the block's scale."""
    s = np.repeat(2.0 ** e.astype(np.float64), 128, axis=1)[:, :x.shape[1]]
    return np.maximum(np.abs(x) * 2.0 ** -4, s * 2.0 ** -10)


@pytest.mark.parametrize("T,H", [(1, 1), (77, 2), (320, 4)])
def test_forward(T, H):
    x, w, scale, shift, pos = _inputs(T, H, T)
    D = H * 128
    W = kl.quantize_fp8_block(w, "tile")
    y, mean, rstd, before, qkv, att = _layer(x, W, scale, shift, pos, H)
    # every stage from the one before it
    ref = P.layer_norm(_np(x), _np(scale), _np(shift), True)[0]
    assert np.all(np.abs(_np(y) - ref) <= np.abs(ref) * 2.0 ** -8 + 1e-4 * np.abs(ref).max())
    ye = P.fp8_encode(_np(y))
    we = P.fp8_encode(_np(w), "tile")
    prod = P.fp8_decode(*ye) @ P.fp8_decode(*we).T
    mag = np.abs(P.fp8_decode(*ye)) @ np.abs(P.fp8_decode(*we)).T
    tol = (D // 32 + 33) * 2.0 ** -23 * mag
    assert np.all(np.abs(_np(before) - prod) <= tol * 1.01 + np.abs(prod) * 2.0 ** -8)
    heads = _np(before).reshape(T, 3 * H, 128)
    rot = P.rope_axes(heads[:, :2 * H], pos.cpu().numpy(), SECTIONS)
    got = _np(qkv).reshape(T, 3 * H, 128)
    assert np.all(np.abs(got[:, :2 * H] - rot) <= np.abs(rot) * 2.0 ** -8 + 2e-6 * np.abs(heads).max())
    np.testing.assert_array_equal(got[:, 2 * H:], heads[:, 2 * H:])
    a, _ = block.attention(*(got[:, i * H:(i + 1) * H] for i in range(3)))
    assert rel_l2(_np(att).reshape(T, H, 128), a) <= 1e-2  # the attention's own tests' bound
    # and the encoded product against the unencoded one: within what the codes may be off by
    ye2, we2 = _encode_error(_np(y), ye[1]), _encode_error(_np(w), we[1])
    full = _np(y) @ _np(w).T
    bound = ye2 @ np.abs(_np(w)).T + np.abs(_np(y)) @ we2.T + ye2 @ we2.T
    assert np.all(np.abs(_np(before) - full) <= bound + tol * 1.01 + np.abs(_np(before)) * 2.0 ** -8)
    assert kl.device_status() == "KL_OK"


def test_forward_captured_and_on_another_stream():
    x, w, scale, shift, pos = _inputs(200, 2, 7)
    W = kl.quantize_fp8_block(w, "tile")
    want = [_layer(x * k, W, scale, shift, pos, 2) for k in (1.0, 0.5)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = _layer(x, W, scale, shift, pos, 2)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want[0]))
    buf = x.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = _layer(buf, W, scale, shift, pos, 2)
    for k, ref in ((0.5, want[1]), (1.0, want[0]), (0.5, want[1])):
        buf.copy_(x * k)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, ref))


@pytest.mark.parametrize("T,H", [(33, 1), (300, 2)])
def test_backward(T, H):
    x, w, scale, shift, pos = _inputs(T, H, T + 1)
    D = H * 128
    y, mean, rstd = kl.layer_norm_forward(x, scale, shift, modulate=True)
    g = torch.Generator().manual_seed(T)
    dout = torch.randn(T, 3 * D, generator=g).bfloat16().cuda()
    # through the rotation of q and k: the inverse rotation of their gradients
    dqkv = dout.clone()
    dqk = dqkv.view(T, 3 * H, 128)[:, :2 * H]
    kl.rope_axes(dqk, pos, SECTIONS, inverse=True, out=dqk)
    ref = P.rope_axes(_np(dout).reshape(T, 3 * H, 128)[:, :2 * H], pos.cpu().numpy(), SECTIONS, inverse=True)
    assert np.all(np.abs(_np(dqk) - ref) <= np.abs(ref) * 2.0 ** -8 + 2e-6 * np.abs(_np(dout)).max())
    # dy = dqkv W and dW = dqkv^T y from transposed encodings
    dy = kl.gemm_fp8_block(kl.quantize_fp8_block(dqkv), kl.quantize_fp8_block(w, "tile", transpose=True))
    dw = kl.gemm_fp8_block(kl.quantize_fp8_block(dqkv, transpose=True), kl.quantize_fp8_block(y, transpose=True),
                           out_dtype=torch.float32)
    for got, (a, ab), (b, bb) in ((dy, (_np(dqkv), "row"), (_np(w).T, "tile")),
                                  (dw, (_np(dqkv).T, "row"), (_np(y).T, "row"))):
        ae, be = _encode_error(a, P.block_exponents(a, ab)), _encode_error(b, P.block_exponents(b, bb))
        full = a @ b.T
        sums = (a.shape[1] // 32 + 34) * 2.0 ** -23 * ((np.abs(a) + ae) @ (np.abs(b) + be).T)
        bound = ae @ np.abs(b).T + np.abs(a) @ be.T + ae @ be.T + sums
        step = 2.0 ** -8 if got.dtype == torch.bfloat16 else 2.0 ** -24
        assert np.all(np.abs(_np(got) - full) <= bound + np.abs(_np(got)) * step)
    # the LayerNorm's gradients from dy, and a directional difference of the layer norm itself
    dx, dscale, dshift = kl.layer_norm_backward(dy, x, mean, rstd, scale, modulate=True)
    rx, rg, rb = P.layer_norm_backward(_np(dy), _np(x), _np(mean), _np(rstd), _np(scale), True, 1)
    for got, r in ((dx, rx), (dscale, rg), (dshift, rb)):
        assert rel_l2(_np(got), r) <= (2.0 ** -8 if got.dtype == torch.bfloat16 else 1e-5)
    u = np.random.default_rng(0).standard_normal(x.shape)
    f = lambda X: (P.layer_norm(X, _np(scale), _np(shift), True)[0] * _np(dy)).sum()
    h = 1e-5
    diff = (f(_np(x) + h * u) - f(_np(x) - h * u)) / (2 * h)
    # bf16 dx: each term off by 2^-8 of itself; the saved statistics are fp32
    assert abs(diff - (_np(dx) * u).sum()) <= (np.abs(_np(dx) * u) * 2.0 ** -8).sum() + 1e-4 * np.abs(rx * u).sum()
    assert kl.device_status() == "KL_OK"


def test_first_calls_of_a_process_captured():
    # nothing is loaded, queried or set up in a way that a capture forbids
    code = """
import torch, diffusion_transformer_image_nvfp4_b200 as kl
def captured(f):
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        r = f()
    g.replay()
    torch.cuda.synchronize()
    return r
def same(a, b):
    assert all(torch.equal(i, j) for i, j in zip(a, b))
x, w = (torch.randn(n, 1328, device="cuda").bfloat16() for n in (3000, 1000))
W = captured(lambda: kl.quantize_fp8_block(w, "tile"))
for rows in (1, 333, 3000):
    A = captured(lambda: kl.quantize_fp8_block(x[:rows]))
    same([captured(lambda: kl.gemm_fp8_block(A, W))], [kl.gemm_fp8_block(A, W)])
for rows in (10, 3000):
    f = captured(lambda: kl.layer_norm_forward(x[:rows]))
    same(f, kl.layer_norm_forward(x[:rows]))
    b = lambda: kl.layer_norm_backward(x[:rows], x[:rows], f[1], f[2])
    same(captured(b), b())
h, pos = x[:, None, :512], torch.arange(3000, device="cuda")[:, None]
same([captured(lambda: kl.rope_axes(h, pos, (256,)))], [kl.rope_axes(h, pos, (256,))])
assert kl.device_status() == "KL_OK"
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=240,
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert r.returncode == 0, r.stdout + r.stderr
