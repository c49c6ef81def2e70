"""CPU-only checks of the eight-bit projection path's entry points: sizes, and
what each refuses before any device work."""

import ctypes

import pytest
import torch

import diffusion_transformer_image_nvfp4_b200 as kl
from diffusion_transformer_image_nvfp4_b200 import build

FAKE = 1 << 20  # never dereferenced: every call below fails its checks first
INVALID, SHAPE, MISALIGNED, WORKSPACE = 1, 2, 3, 4


@pytest.fixture(scope="module")
def L():
    build.build()
    return kl.lib()


def test_fp8_scale_sizes(L):
    mma, tile = kl.KL_SCALE_MMA, kl.KL_FP8_TILE
    assert L.kl_fp8_scales_bytes(1, 1, mma) == 512
    assert L.kl_fp8_scales_bytes(129, 513, mma) == 2 * 2 * 512
    assert L.kl_fp8_scales_bytes(129, 513, mma | tile) == 2 * 2 * 512
    assert L.kl_fp8_scales_bytes(129, 513, 0) == 129 * 5
    assert L.kl_fp8_scales_bytes(129, 513, tile) == 2 * 5
    assert L.kl_fp8_scales_bytes(-1, 5, 0) == 0


def test_quantize_refusals(L):
    def q(x=FAKE, dt=0, r=4, c=64, ldx=64, codes=FAKE, ldc=64, sc=FAKE, flags=1):
        return L.kl_quantize_fp8_block(x, dt, r, c, ldx, codes, ldc, sc, flags, None)

    assert q(x=None) == q(codes=None) == q(sc=None) == INVALID
    assert q(dt=3) == q(dt=-1) == INVALID
    assert q(flags=2) == q(flags=64) == INVALID
    assert q(r=0) == q(c=0) == q(r=1 << 31) == SHAPE
    assert q(r=1 << 30, c=1 << 20, ldx=1 << 20, ldc=1 << 20) == SHAPE      # tiles
    assert q(ldx=63) == q(ldc=48) == q(ldc=72) == INVALID
    assert q(ldc=16, flags=1 | kl.KL_FP8_TRANSPOSE, r=17) == INVALID        # 17 encoded columns need 32 bytes
    assert q(x=FAKE + 1) == q(codes=FAKE + 8) == q(sc=FAKE + 2) == MISALIGNED
    assert q(x=FAKE + 2, dt=1) == MISALIGNED


def test_gemm_refusals(L):
    def g(M=4, N=8, K=32, a=FAKE, w=FAKE, sa=FAKE, lda=32, ldw=32, out=FAKE, dt=0, ldo=8, kern=0):
        A, W = kl._FP8Tensor(a, sa, lda), kl._FP8Tensor(w, FAKE, ldw)
        return L.kl_gemm_fp8_block(ctypes.byref(A), ctypes.byref(W), M, N, K, out, dt, ldo, kern, None)

    assert g(a=None) == g(sa=None) == g(out=None) == INVALID
    assert L.kl_gemm_fp8_block(None, None, 4, 8, 32, FAKE, 0, 8, 0, None) == INVALID
    assert g(dt=2) == g(kern=4) == g(kern=-1) == INVALID
    assert g(M=0) == g(N=0) == g(K=0) == g(M=(1 << 30) + 1) == SHAPE
    assert g(M=1 << 30, N=1 << 30, ldo=1 << 30) == SHAPE
    assert g(lda=16) == g(lda=40) == g(ldw=24) == g(ldo=7) == INVALID
    assert g(a=FAKE + 8) == g(w=FAKE + 1) == g(sa=FAKE + 4) == g(out=FAKE + 1) == MISALIGNED
    assert g(out=FAKE + 2, dt=1) == MISALIGNED


def test_rope_refusals(L):
    def r(**kw):
        a = kl._RopeArgs(FAKE, FAKE, FAKE, 0, 0, 0, 0, 3, (ctypes.c_int64 * 4)(16, 24, 24, 0), 1, 8, 2, 128,
                         (ctypes.c_int64 * 3)(0, 256, 128), (ctypes.c_int64 * 3)(0, 256, 128), 10000.0)
        for k, v in kw.items():
            setattr(a, k, (ctypes.c_int64 * 4)(*v) if k == "sections" else v)
        return L.kl_rope_axes(ctypes.byref(a), None)

    assert L.kl_rope_axes(None, None) == INVALID
    assert r(x=None) == r(out=None) == r(pos=None) == INVALID
    assert r(dtype=3) == r(pos_type=3) == r(flags=8) == INVALID
    assert r(theta=1.0) == r(theta=float("nan")) == r(theta=float("inf")) == INVALID
    assert r(naxes=0) == r(naxes=5) == SHAPE
    assert r(sections=(16, 24, 25, 0)) == r(sections=(0, 0, 0, 0)) == r(sections=(-1, 24, 24, 0)) == SHAPE
    assert r(dim=514) == r(dim=127) == r(tokens=0) == r(heads=0) == r(batch=0) == SHAPE
    assert r(batch=1 << 20, tokens=1 << 20) == SHAPE
    def st(*v):
        return (ctypes.c_int64 * 3)(*v)

    # (x is out here) in place at other strides; an output that is broadcast
    assert r(out_stride=st(0, 256, 127)) == r(x_stride=st(0, 0, 128)) == INVALID
    assert r(out=2 * FAKE, out_stride=st(0, 256, 100)) == r(out=2 * FAKE, out_stride=st(0, -127, 128)) == INVALID
    assert r(out=2 * FAKE, out_stride=st(0, 0, 128)) == r(out=2 * FAKE, batch=2, out_stride=st(0, 256, 128)) == INVALID
    assert r(x=FAKE + 1) == r(out=FAKE + 1) == r(pos=FAKE + 2) == r(pos=FAKE + 4, pos_type=1) == MISALIGNED


def test_layer_norm_refusals(L):
    def f(x=FAKE, dt=0, r=6, c=10, ldx=10, gain=None, bias=None, pd=0, groups=1, eps=1e-6, flags=0, y=FAKE, ldy=10,
          mean=None, rstd=None):
        return L.kl_layer_norm_forward(x, dt, r, c, ldx, gain, bias, pd, groups, eps, flags, y, ldy, mean, rstd, None)

    assert f(x=None) == f(y=None) == f(eps=-1.0) == f(eps=float("nan")) == INVALID
    assert f(dt=5) == f(pd=5) == f(flags=2) == f(ldx=9) == f(ldy=9) == INVALID
    assert f(r=0) == f(c=0) == f(groups=4) == f(groups=0) == f(c=(1 << 24) + 1, ldx=1 << 25, ldy=1 << 25) == SHAPE
    assert f(x=FAKE + 1) == f(gain=FAKE + 1) == f(mean=FAKE + 2) == f(bias=FAKE + 2, pd=1) == MISALIGNED

    assert L.kl_layer_norm_backward_workspace_size(0, 6, 10, 1) == 0      # few rows need none
    need = L.kl_layer_norm_backward_workspace_size(0, 6000, 10, 1)
    assert need >= 2 * 10 * 4 and L.kl_layer_norm_backward_workspace_size(0, 6000, 10, 7) == 0
    for dt in (0, 1, 2):   # every width has a size, a single column among them
        for c in (1, 3, 7, 8, 4096, 4097, 1 << 24):
            for g in (1, 5, 100):
                assert L.kl_layer_norm_backward_workspace_size(dt, 60000, c, g) >= g * 2 * c * 4

    def b(dy=FAKE, x=FAKE, ld=10, mean=FAKE, rstd=FAKE, dx=2 * FAKE, dg=FAKE, db=FAKE, ws=FAKE, n=need, groups=1):
        return L.kl_layer_norm_backward(dy, ld, x, 10, 0, 6000, 10, mean, rstd, None, 0, groups, 0, dx, 10, dg, db, ws, n,
                                        None)

    assert b(dy=None) == b(x=None) == b(mean=None) == b(rstd=None) == b(dx=None) == INVALID
    assert b(dg=None) == b(db=None) == INVALID                # both or neither
    assert b(dx=FAKE) == INVALID                              # dx is dy or x
    assert b(ld=9) == INVALID and b(groups=7) == SHAPE
    assert b(ws=None) == b(n=need - 1) == WORKSPACE
    assert b(ws=FAKE + 8) == b(dx=2 * FAKE + 1) == b(dg=FAKE + 2) == MISALIGNED


def test_binding_refuses_cpu_tensors_and_overlapping_rows():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    for call in (lambda: kl.quantize_fp8_block(x), lambda: kl.layer_norm_forward(x),
                 lambda: kl.layer_norm_backward(x, x, x, x),
                 lambda: kl.rope_axes(x.view(4, 1, 64), torch.zeros(4, 1), [32])):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    assert kl._rows(torch.zeros(6, 5, 8), "x") == (30, 8, 8)
    assert kl._rows(torch.zeros(6, 5, 8)[:, :, :3], "x") == (30, 3, 8)
    assert kl._rows(torch.zeros(6, 5, 8)[:, 2, :], "x") == (6, 8, 40)
    assert kl._rows(torch.zeros(6, 5, 8)[:, 2:3, 1:4], "x") == (6, 3, 40)
    assert kl._rows(torch.zeros(7), "x") == (1, 7, 7)
    for bad in (torch.zeros(6, 5, 8)[:, :4], torch.zeros(6, 8).t(), torch.zeros(1, 8).expand(6, 8),
                torch.zeros(0, 8), torch.zeros(())):
        with pytest.raises(ValueError):
            kl._rows(bad, "x")
