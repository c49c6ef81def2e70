"""kl_rope_axes refuses an output whose heads overlap, whichever strides bring
them together, and no other.  (x is misaligned throughout, so a call whose
strides are taken ends there: nothing is ever launched.)"""

import ctypes
import itertools
import random

import pytest
import torch

import diffusion_transformer_image_nvfp4_b200 as kl
from diffusion_transformer_image_nvfp4_b200 import build

FAKE = 1 << 20
INVALID, MISALIGNED = 1, 3


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


def _call(size, stride, dim):
    a = kl._RopeArgs(FAKE + 1, 2 * FAKE, FAKE, 0, 0, 0, 0, 1, (ctypes.c_int64 * 4)(dim // 2, 0, 0, 0), *size, dim,
                     (ctypes.c_int64 * 3)(0, dim, 0), (ctypes.c_int64 * 3)(*stride), 10000.0)
    return kl.lib().kl_rope_axes(ctypes.byref(a), None)


def _overlaps(size, stride, dim):
    at = sorted(sum(i * s for i, s in zip(ix, stride)) for ix in itertools.product(*map(range, size)))
    return any(b - a < dim for a, b in zip(at, at[1:]))


def test_strides_that_collide_only_together():
    assert _call((1, 2, 3), (0, 8, 8), 8) == INVALID      # (t 0, h 1) is (t 1, h 0)
    assert _call((2, 1, 3), (8, 0, 8), 8) == INVALID      # batch and head
    assert _call((2, 3, 1), (8, 8, 0), 8) == INVALID      # batch and token
    assert _call((1, 4, 4), (0, 24, 8), 8) == INVALID     # the fourth head is the next token's first
    assert _call((1, 4, 3), (0, 24, 8), 8) == MISALIGNED
    assert _call((2, 4, 3), (56, 16, 24), 8) == INVALID
    assert _call((1, 5, 2), (0, 24, 16), 8) == MISALIGNED  # 0, 24, ... 96 and 16, 40, ...: interleaved, apart
    assert _call((1, 2, 3), (0, -8, 8), 8) == INVALID


@pytest.mark.parametrize("dim", [2, 6])
def test_every_small_layout(dim):
    r = random.Random(dim)
    seen = {INVALID: 0, MISALIGNED: 0}
    for _ in range(6000):
        size = tuple(r.randint(1, 6) for _ in range(3))
        stride = tuple(r.choice((-1, 1)) * r.randint(0, 14 * dim) for _ in range(3))
        want = INVALID if _overlaps(size, stride, dim) else MISALIGNED
        assert _call(size, stride, dim) == want, (size, stride)
        seen[want] += 1
    assert min(seen.values()) > 500


def test_ordinary_layouts_of_any_size_are_taken():
    for size in ((3, 4600, 20), (1, 1 << 20, 40), (1 << 10, 1 << 10, 24)):
        d = 128
        for order in itertools.permutations(range(3)):
            stride, span = [0, 0, 0], d
            for i in order:
                stride[i], span = span, span * size[i]
            assert _call(size, stride, d) == MISALIGNED
    top = (1 << 63) - 1
    assert _call((2, 2, 2), (top, 1 << 40, 128), 128) == MISALIGNED
    assert _call((2, 2, 2), (-top - 1, 1 << 40, 128), 128) == INVALID
    # collisions among very many heads are refused too, unsearched
    assert _call((1 << 10, 1 << 10, 1 << 10), (130, 131, 132), 128) == INVALID


@pytest.mark.gpu
def test_colliding_outputs_are_refused_in_python():
    x = torch.randn(2, 3, 8, device="cuda")
    pos = torch.zeros(2, 1, dtype=torch.int32, device="cuda")
    buf = torch.zeros(64, device="cuda")
    with pytest.raises(kl.KLError, match="INVALID_ARG"):
        kl.rope_axes(x, pos, (4,), out=buf.as_strided((2, 3, 8), (8, 8, 1)))
    assert (buf == 0).all()
    apart = buf.as_strided((2, 3, 8), (8, 16, 1))  # interleaved: the heads of a token with the next one's between
    assert torch.equal(kl.rope_axes(x, pos, (4,), out=apart), x)
