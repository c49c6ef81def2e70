"""FP8 encode and product (kl_quantize_fp8_block, kl_gemm_fp8_block) against
the fp64 definitions."""

import ctypes

import numpy as np
import pytest
import torch

import diffusion_transformer_image_nvfp4_b200 as kl
from oracle import projection as P

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def _x(shape, seed, std=1.0, dtype=torch.float32):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(*shape, generator=g) * std
    x *= torch.exp2(torch.randint(-6, 7, (shape[0], 1), generator=g).float())
    return x.to(dtype)


def _np(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def _encoded(x, block, transpose):
    return P.fp8_encode(_np(x).T if transpose else _np(x), block)


def _check_encode(x, q, block, transpose):
    codes, e = _encoded(x, block, transpose)
    got = q.codes.cpu().numpy()
    np.testing.assert_array_equal(got[:, :codes.shape[1]], codes)
    assert not got[:, codes.shape[1]:].any()
    if q.layout == "mma":
        np.testing.assert_array_equal(q.scales.cpu().numpy(), P.scales_mma(e))
    else:
        np.testing.assert_array_equal(q.scales.cpu().numpy(), (e[::128] if block == "tile" else e) + 127)


@pytest.mark.parametrize("shape", [(1, 1), (1, 128), (3, 17), (5, 512), (128, 128), (130, 700), (257, 1040), (300, 513)])
@pytest.mark.parametrize("block,transpose", [("row", False), ("row", True), ("tile", False), ("tile", True)])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_encode_bit_exact(shape, block, transpose, dtype):
    x = _x(shape, sum(shape), dtype=DT[dtype]).cuda()
    for layout in ("mma", "linear"):
        _check_encode(x, kl.quantize_fp8_block(x, block, transpose, layout), block, transpose)
    assert kl.device_status() == "KL_OK"


@pytest.mark.parametrize("block,transpose", [("row", False), ("row", True), ("tile", False)])
def test_encode_edges(block, transpose):
    # exact borders of the scale, zeros, the least and the largest values, ties
    x = torch.zeros(256, 256)
    x[0, 0], x[1, 0], x[2, 0] = 448.0, 448.00003, 2.0 ** -149
    x[3, 0], x[4, 0], x[5, :128] = 3.4028234e38, -1.75, 1.0
    x[5, 64:128] = 17.0 / 16 * 2.0 ** -7         # halfway between two E4M3 values
    x[200, 130], x[201, 140] = 2.0 ** -126, -0.0
    x = x.cuda()
    _check_encode(x, kl.quantize_fp8_block(x, block, transpose), block, transpose)
    assert kl.device_status() == "KL_OK"


def test_encode_strided_rows_batches_and_misaligned():
    big = _x((40, 1000), 3, dtype=torch.bfloat16).cuda()
    for view in (big[:, 5:305], big[3:20, 8:520], big[:, :1], big.view(10, 4, 1000)[:, 1, 16:400],
                 big.view(10, 4, 1000)[..., :640]):
        flat = view.reshape(-1, view.shape[-1])
        for block, tr in (("row", False), ("row", True), ("tile", False)):
            _check_encode(flat, kl.quantize_fp8_block(view, block, tr), block, tr)


def test_encode_nonfinite_blocks_become_nan_and_are_recorded():
    x = _x((256, 512), 4).cuda()
    x[3, 130], x[200, 5] = float("nan"), float("-inf")
    assert kl.device_status() == "KL_OK"
    q = kl.quantize_fp8_block(x, layout="linear")
    s = q.scales.cpu().numpy()
    assert s[3, 1] == 255 and s[200, 0] == 255 and (s == 255).sum() == 2
    c = q.codes.cpu().numpy()
    assert (c[3, 128:256] == 0x7F).all() and (c[200, :128] == 0x7F).all()
    ok = x.clone()
    ok[3, 130] = ok[200, 5] = 0
    clean = kl.quantize_fp8_block(ok, layout="linear").codes.cpu().numpy()
    np.testing.assert_array_equal(np.delete(c, [3, 200], 0), np.delete(clean, [3, 200], 0))
    assert kl.device_status() == "KL_ERR_NONFINITE"
    for block, tr in (("tile", False), ("row", True), ("tile", True)):
        s = kl.quantize_fp8_block(x, block, tr, "linear").scales
        assert int((s == 255).sum()) == 2
        assert kl.device_status() == "KL_ERR_NONFINITE"
    # a NaN block makes its outputs NaN and no others
    q = kl.quantize_fp8_block(x)
    y = kl.gemm_fp8_block(q, kl.quantize_fp8_block(_x((64, 512), 5).cuda(), "tile"))
    bad = torch.isnan(y).all(1).cpu()
    assert bad[3] and bad[200] and bad.sum() == 2 and torch.isnan(y).sum() == 2 * 64
    kl.device_status()


@pytest.mark.parametrize("R,C", [(6000, 4200), (40000, 600), (1500, 20000), (129, 100003)])
def test_encode_large_equals_its_parts(R, C):
    # several words and rows a warp, several tiles a column: as encoded a part at a time
    x = _x((R, C), R, dtype=torch.bfloat16).cuda()
    q = kl.quantize_fp8_block(x)
    for r in (0, 1, R // 2, R - 1):
        part = kl.quantize_fp8_block(x[r:r + 1])
        _check_encode(x[r:r + 1], part, "row", False)
        assert torch.equal(q.codes[r], part.codes[0])
    lin = kl.quantize_fp8_block(x, layout="linear")
    assert torch.equal(lin.codes, q.codes)
    s = kl.quantize_fp8_block(x[128:256], layout="linear").scales
    assert torch.equal(lin.scales[128:256], s)
    t = kl.quantize_fp8_block(x, transpose=True, layout="linear")
    for c in (0, C // 2, C - 1):
        part = kl.quantize_fp8_block(x[:, c:c + 1].t().contiguous(), layout="linear")
        assert torch.equal(t.codes[c, :R], part.codes[0, :R]) and torch.equal(t.scales[c], part.scales[0])
    tile = kl.quantize_fp8_block(x, "tile", layout="linear")
    last = kl.quantize_fp8_block(x[(R - 1) // 128 * 128:], "tile", layout="linear")
    assert torch.equal(tile.scales[-1:], last.scales) and torch.equal(tile.codes[-last.rows:], last.codes)
    tt = kl.quantize_fp8_block(x, "tile", transpose=True, layout="linear")
    assert torch.equal(tt.scales, tile.scales.t()) and torch.equal(tt.codes[:, :R], tile.codes[:, :C].t())
    assert kl.device_status() == "KL_OK"


def test_codes_past_the_last_column_are_zero_in_nan_blocks_too():
    x = torch.full((20, 37), float("nan"), device="cuda")
    for block, tr in (("row", False), ("row", True), ("tile", False), ("tile", True)):
        q = kl.quantize_fp8_block(x, block, tr)
        assert (q.codes[:, :q.cols] == 0x7F).all() and not q.codes[:, q.cols:].any()
    assert kl.device_status() == "KL_ERR_NONFINITE"


@pytest.mark.parametrize("off", range(0, 9))
def test_encode_rows_at_every_alignment(off):
    # rows start at every 16-bit and 32-bit offset within 16 bytes; the matrix ends with its buffer
    for dtype, cols in ((torch.bfloat16, 77), (torch.float16, 530), (torch.float32, 1041)):
        x = _x((9, cols + 3), off, dtype=dtype).cuda().flatten()[off:]
        x = x[:(x.numel() // (cols + 2)) * (cols + 2)].view(-1, cols + 2)[:, 2:]
        for block in ("row", "tile"):
            _check_encode(x, kl.quantize_fp8_block(x, block), block, False)


def test_encode_leaves_what_is_past_the_padded_columns():
    x = _x((5, 20), 6).cuda()
    codes = torch.full((5, 64), 0xAB, dtype=torch.uint8, device="cuda")
    scales = torch.empty(512, dtype=torch.uint8, device="cuda")
    st = kl.lib().kl_quantize_fp8_block(x.data_ptr(), 1, 5, 20, 20, codes.data_ptr(), 64, scales.data_ptr(),
                                        kl.KL_SCALE_MMA, torch.cuda.current_stream().cuda_stream)
    assert st == 0
    c = codes.cpu().numpy()
    assert (c[:, 32:] == 0xAB).all() and (c[:, 20:32] == 0).all()


# ------------------------------------------------------------------ product
def _operands(M, N, K, seed, w_block="tile"):
    a, w = _x((M, K), seed).cuda(), _x((N, K), seed + 1, 0.02).cuda()
    return a, w, kl.quantize_fp8_block(a), kl.quantize_fp8_block(w, w_block)


def _check_product(got, a, w, K, bf16, w_block="tile"):
    """Every partial sum is held in fp32: an instruction adds 32 exact products
    to the sum with at most 33 roundings or truncations of one unit (2^-23) of
    its largest term, which is at most the sum of the magnitudes; a bf16 result
    is off by half a step more."""
    A, W = P.fp8_decode(*P.fp8_encode(a)), P.fp8_decode(*P.fp8_encode(w, w_block))
    ref, mag = A @ W.T, np.abs(A) @ np.abs(W).T
    tol = (-(-K // 32) + 33) * 2.0 ** -23 * mag + 1e-38
    if bf16:
        tol = tol * (1 + 2.0 ** -8) + np.abs(ref) * 2.0 ** -8
    d = np.abs(got - ref)
    assert np.all(d <= tol), (d / tol).max()


KERNELS = ["auto", "pair_256x256", "pair_256x128", "split"]


# one token to several tiles; K of one group, of part of one, of a block and a
# bit, past one and several scale atoms; odd N (rows that are not aligned)
@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("M,N,K", [(1, 1, 1), (1, 128, 128), (3, 130, 40), (16, 256, 513), (17, 96, 160),
                                   (33, 1000, 1328), (65, 129, 600), (128, 512, 2048), (129, 257, 130),
                                   (300, 520, 1100), (520, 264, 4224)])
def test_product(M, N, K, kernel):
    a, w, A, W = _operands(M, N, K, M + N + K)
    for dt in (torch.float32, torch.bfloat16):
        got = kl.gemm_fp8_block(A, W, out_dtype=dt, kernel=kernel)
        _check_product(_np(got), _np(a), _np(w), K, dt == torch.bfloat16)
    assert kl.device_status() == "KL_OK"


@pytest.mark.parametrize("kernel", ["auto", "split"])
def test_product_many_token_tiles_of_few_rows(kernel):
    # rows of very different scales: a tile that read another's scale bytes would show at once
    for M, N, K in ((40, 128, 300), (100, 1000, 256), (200, 96, 1300), (333, 1000, 1328), (1000, 128, 640)):
        a, w, A, W = _operands(M, N, K, M, "row")
        got = kl.gemm_fp8_block(A, W, out_dtype=torch.float32, kernel=kernel)
        _check_product(_np(got), _np(a), _np(w), K, False, "row")
    assert kl.device_status() == "KL_OK"


@pytest.mark.parametrize("split_rows", [1, 40])
def test_product_same_bits_every_run(split_rows):
    _, _, A, W = _operands(split_rows, 384, 3000, 5)
    first = kl.gemm_fp8_block(A, W, out_dtype=torch.float32)
    for _ in range(3):
        assert torch.equal(first, kl.gemm_fp8_block(A, W, out_dtype=torch.float32))


@pytest.mark.parametrize("M", [1, 200, 700])
def test_product_writes_a_strided_view_and_nothing_else(M):
    a, w, A, W = _operands(M, 200, 300, 9)
    for dt in (torch.bfloat16, torch.float32):
        for off, ld in ((0, 256), (3, 209), (8, 240)):
            buf = torch.full((M + 2, ld), 7.0, dtype=dt, device="cuda")
            view = buf[1:M + 1, off:off + 200]
            for kernel in KERNELS:
                buf.fill_(7.0)
                kl.gemm_fp8_block(A, W, out=view, kernel=kernel)
                _check_product(_np(view), _np(a), _np(w), 300, dt == torch.bfloat16)
                assert (buf[0] == 7).all() and (buf[-1] == 7).all()
                assert (buf[:, :off] == 7).all() and (buf[:, off + 200:] == 7).all()


def test_product_of_row_encoded_weights_and_wider_buffers():
    a, w, A, W = _operands(70, 150, 260, 11, "row")
    wide = torch.full((70, 288), 0x7F, dtype=torch.uint8, device="cuda")  # NaN codes past K are never read
    wide[:, :260] = A.codes[:, :260]
    A2 = kl.FP8Block(wide, A.scales, 70, 260)
    for kernel in KERNELS:
        got = kl.gemm_fp8_block(A2, W, out_dtype=torch.float32, kernel=kernel)
        _check_product(_np(got), _np(a), _np(w), 260, False, "row")


def test_whole_numbers_are_exact():
    # products of small whole numbers sum exactly in fp32: any wrong scale byte, row or column shows
    g = torch.Generator().manual_seed(1)
    a = torch.randint(-4, 5, (300, 1500), generator=g).float()
    w = torch.randint(-4, 5, (400, 1500), generator=g).float()
    a *= torch.exp2(torch.randint(-3, 4, (300, 1), generator=g).float())
    for kernel in KERNELS:
        got = kl.gemm_fp8_block(kl.quantize_fp8_block(a.cuda()), kl.quantize_fp8_block(w.cuda(), "row"),
                                out_dtype=torch.float32, kernel=kernel)
        np.testing.assert_array_equal(_np(got), _np(a) @ _np(w).T)


def test_product_refusals():
    _, _, A, W = _operands(4, 32, 64, 1)
    lin = kl.quantize_fp8_block(torch.zeros(4, 64, device="cuda"), layout="linear")
    with pytest.raises(ValueError, match="layout"):
        kl.gemm_fp8_block(lin, W)
    with pytest.raises(ValueError, match="share K"):
        kl.gemm_fp8_block(kl.FP8Block(A.codes, A.scales, 4, 48), W)
    with pytest.raises(ValueError, match="too small"):
        kl.gemm_fp8_block(kl.FP8Block(A.codes, A.scales[:256], 4, 64), W)
    with pytest.raises(ValueError, match="codes"):
        kl.gemm_fp8_block(kl.FP8Block(A.codes, A.scales, 5, 64), W)
    with pytest.raises(ValueError, match="out_dtype"):
        kl.gemm_fp8_block(A, W, out_dtype=torch.float16)
    with pytest.raises(ValueError, match="out"):
        kl.gemm_fp8_block(A, W, out=torch.empty(4, 33, device="cuda"))
    with pytest.raises(kl.KLError, match="INVALID_ARG"):
        kl.gemm_fp8_block(kl.FP8Block(A.codes[:, :56].contiguous(), A.scales, 4, 56),
                          kl.FP8Block(W.codes, W.scales, 32, 56))  # row stride 56: not a multiple of 16


def test_streams_and_graph():
    x, w = _x((40, 640), 21).cuda(), _x((96, 640), 22, 0.02).cuda()
    W = kl.quantize_fp8_block(w, "tile")
    want = kl.gemm_fp8_block(kl.quantize_fp8_block(x), W)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = kl.gemm_fp8_block(kl.quantize_fp8_block(x), W)
    side.synchronize()
    assert torch.equal(got, want)
    buf = x.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = kl.gemm_fp8_block(kl.quantize_fp8_block(buf), W)
    for k in (1.0, -2.0, 0.5):
        buf.copy_(x * k)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, kl.gemm_fp8_block(kl.quantize_fp8_block(x * k), W))


def test_many_rows_offset_past_32_bits():
    # 2^31 elements of x, rows far apart: the last row's encoding is the row's own
    rows, cols = 1 << 20, 2064
    x = torch.zeros((rows, cols), dtype=torch.bfloat16, device="cuda")
    x[-1] = _x((1, cols), 23, dtype=torch.bfloat16).cuda()
    q = kl.quantize_fp8_block(x)
    one = kl.quantize_fp8_block(x[-1:])
    assert torch.equal(q.codes[-1], one.codes[0]) and not q.codes[:-1].any()
    del x
    w = kl.quantize_fp8_block(_x((2056, cols), 24, 0.02).cuda(), "tile")
    y = kl.gemm_fp8_block(q, w)  # 2^31 outputs
    y1 = kl.gemm_fp8_block(one, w, kernel="pair_256x256")
    assert torch.equal(y[-1], y1[0]) and not y[:-1].any()
