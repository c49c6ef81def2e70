"""Cases for the eight-bit projection path: block-scaled FP8 encode and product, multi-axis rotary
positions, LayerNorm forward and backward.

``run`` computes an operator in plain torch operations (``own`` false) or through the framework's entry
points (``own`` true).  Sizes are the 1024 x 1024 workloads of this repository (4,608 / 8,704 / 20,992
tokens, width 3,072, 24 heads of 128, MLP 9,216), its small configurations, and generic odd ones.
"""

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
POS = {"i32": torch.int32, "i64": torch.int64, "f32": torch.float32}


def listed():
    return [
        # the MLP's hidden activations of the 1024^2 text-to-image block before the down projection
        dict(name="quantize hidden 4608x9216", op="quantize", rows=4608, cols=9216, dtype="bf16", block="row",
             transpose=False, layout="mma"),
        # an output gradient encoded along its tokens, for a weight gradient; odd sizes, 32-bit values
        dict(name="quantize grad^T 1021x1155", op="quantize", rows=1021, cols=1155, dtype="fp32", block="row",
             transpose=True, layout="mma"),
        # one token through the QKV projection: the weights are read once and that is all the work
        dict(name="gemm one token", op="gemm", m=1, n=9216, k=3072, out="bf16"),
        # a short prompt's rows through a ragged projection, 32-bit results
        dict(name="gemm ragged 333x1000x1328", op="gemm", m=333, n=1000, k=1328, out="fp32"),
        # the text-to-image block's QKV projection
        dict(name="gemm qkv 4608", op="gemm", m=4608, n=9216, k=3072, out="bf16"),
        # the MLP down projection of the four-reference block: the longest batch
        dict(name="gemm down 20992", op="gemm", m=20992, n=3072, k=9216, out="bf16"),
        # q and k of the QKV projection's output, read in place (row stride 3 D), image grid positions
        dict(name="rope qk 4608x48", op="rope", batch=1, tokens=4608, heads=48, spare=24, dim=128, sections="16,24,24",
             dtype="bf16", pairing="interleaved", ladder="axis", pos="i32", inverse=False),
        # gradient through the rotation of two video clips (time, height, width), part of each head, half pairing
        dict(name="rope video grad 2x3315x6", op="rope", batch=2, tokens=3315, heads=6, spare=0, dim=96,
             sections="8,16,16", dtype="fp32", pairing="half", ladder="shared", pos="f32", inverse=True),
        # the text rows of the smallest configuration: latency
        dict(name="ln forward 16x128", op="ln_forward", rows=16, cols=128, groups=1, dtype="bf16", pdtype="bf16",
             affine="modulate"),
        # two images of the image-to-image block with their own modulation
        dict(name="ln forward 2x8704x3072", op="ln_forward", rows=17408, cols=3072, groups=2, dtype="bf16",
             pdtype="bf16", affine="modulate"),
        # gradient of the same step on the four-reference block
        dict(name="ln backward 20992x3072", op="ln_backward", rows=20992, cols=3072, groups=1, dtype="bf16",
             pdtype="bf16", affine="modulate"),
        # an odd small layer norm with an ordinary weight and bias, 32-bit values
        dict(name="ln backward 77x1155", op="ln_backward", rows=77, cols=1155, groups=1, dtype="fp32", pdtype="fp32",
             affine="gain"),
    ]


def _log(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["quantize", "gemm", "gemm", "rope", "ln_forward", "ln_backward"])
    if op == "quantize":
        return dict(op=op, rows=_log(rng, 1, 20992), cols=_log(rng, 1, 2048), dtype=rng.choice(list(DTYPES)),
                    block=rng.choice(["row", "row", "tile"]), transpose=rng.random() < 0.4,
                    layout=rng.choice(["mma", "mma", "linear"]))
    if op == "gemm":
        return dict(op=op, m=_log(rng, 1, 20992), n=_log(rng, 16, 9216), k=_log(rng, 32, 3072),
                    out=rng.choice(["bf16", "bf16", "fp32"]))
    if op == "rope":
        axes = rng.randint(1, 4)
        sections = [rng.randint(1, 24) for _ in range(axes)]
        dim = max(2 * sum(sections) + 2 * rng.randint(0, 8), 8)
        return dict(op=op, batch=rng.randint(1, 3), tokens=_log(rng, 1, 4608), heads=rng.randint(1, 24),
                    spare=rng.choice([0, 0, 3]), dim=dim, sections=",".join(map(str, sections)),
                    dtype=rng.choice(list(DTYPES)), pairing=rng.choice(["interleaved", "half"]),
                    ladder=rng.choice(["axis", "shared"]), pos=rng.choice(list(POS)), inverse=rng.random() < 0.5)
    groups = rng.choice([1, 1, 2, 3])
    return dict(op=op, rows=groups * _log(rng, 1, 5000), cols=_log(rng, 16, 4096), groups=groups,
                dtype=rng.choice(list(DTYPES)), pdtype=rng.choice(["same", "fp32"]),
                affine=rng.choice(["modulate", "gain", "none"]))


def work(case):
    op = case["op"]
    if op == "quantize":
        r, c, es = case["rows"], case["cols"], DTYPES[case["dtype"]].itemsize
        blocks = (r * c / 128.0) if case["block"] == "row" or case["layout"] == "mma" else (r * c / 16384.0)
        return {"bytes": r * c * (es + 1) + blocks, "flops": 3.0 * r * c}
    if op == "gemm":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": (m + n) * k * (1 + 1 / 128.0) + m * n * DTYPES[case["out"]].itemsize, "flops": 2.0 * m * n * k}
    if op == "rope":
        n = case["batch"] * case["tokens"] * case["heads"] * case["dim"]
        return {"bytes": 2.0 * n * DTYPES[case["dtype"]].itemsize, "flops": 3.0 * n}
    n, es = case["rows"] * case["cols"], DTYPES[case["dtype"]].itemsize
    if op == "ln_forward":
        return {"bytes": 2.0 * n * es + 8.0 * case["rows"], "flops": 8.0 * n}
    return {"bytes": 3.0 * n * es + 8.0 * case["rows"], "flops": 14.0 * n}


# ------------------------------------------------------------------ inputs
def _activations(gen, rows, cols, dtype):
    """Normal values with a spread of magnitudes over rows and a few strong columns, as activations have."""
    x = torch.randn(rows, cols, generator=gen, device="cuda")
    x *= torch.exp(0.5 * torch.randn(rows, 1, generator=gen, device="cuda"))
    strong = torch.rand(1, cols, generator=gen, device="cuda") < 0.01
    return torch.where(strong, 12.0 * x, x).to(dtype)


def _pow2(e):
    """2^e in 32 bits for whole e in [-127, 127] (2^-127 is below the normal range)."""
    normal = ((e.clamp(min=-126) + 127) << 23).view(torch.float32)
    return torch.where(e < -126, normal * 0.5, normal)


def _mma_scales(s):
    """Scale bytes [rows, blocks] in 512-byte atoms of 128 rows x 4 blocks; what is past the end is 0."""
    r, b = s.shape
    rp, bp = -(-r // 128) * 128, -(-b // 4) * 4
    full = torch.zeros(rp, bp, dtype=torch.uint8, device=s.device)
    full[:r, :b] = s
    return full.view(rp // 128, 4, 32, bp // 4, 4).permute(0, 3, 2, 1, 4).reshape(-1)


def _linear_scales(flat, rows, cols):
    b = -(-cols // 128)
    a = flat.view(-(-rows // 128), -(-b // 4), 32, 4, 4).permute(0, 3, 2, 1, 4)
    return a.reshape(-(-rows // 128) * 128, -1)[:rows, :b]


def _encode(x, block):
    """(codes uint8 [rows, cols padded to 16], scale bytes [rows or row tiles, blocks]) of x in 32 bits."""
    r, c = x.shape
    nb = -(-c // 128)
    p = torch.zeros(r, nb * 128, device=x.device)
    p[:, :c] = x
    amax = p.view(r, nb, 128).abs().amax(2)
    if block == "tile":
        rt = -(-r // 128)
        t = torch.zeros(rt * 128, nb, device=x.device)
        t[:r] = amax
        tiles = t.view(rt, 128, nb).amax(1)
        amax = tiles.repeat_interleave(128, 0)[:r]
    frac, ex = torch.frexp(amax)  # amax = frac 2^ex, frac in [1/2, 1); 448 = 0.875 2^9
    e = (ex - 9 + (frac > 0.875).int()).clamp(-127, 127)
    e = torch.where(amax == 0, torch.zeros_like(e), e)
    q = (p.view(r, nb, 128) * _pow2(-e)[:, :, None]).view(r, nb * 128).to(torch.float8_e4m3fn)
    codes = q.view(torch.uint8)[:, :-(-c // 16) * 16].contiguous()
    return codes, (e + 127).to(torch.uint8)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    if op == "quantize":
        return case, _activations(gen, case["rows"], case["cols"], DTYPES[case["dtype"]])
    if op == "gemm":
        m, n, k = case["m"], case["n"], case["k"]
        a, sa = _encode(_activations(gen, m, k, torch.float32), "row")
        w, sw = _encode(0.02 * torch.randn(n, k, generator=gen, device="cuda"), "tile")
        return case, a, _mma_scales(sa), w, _mma_scales(sw)
    if op == "rope":
        b, t, h, d = case["batch"], case["tokens"], case["heads"], case["dim"]
        buf = torch.randn(b, t, h + case["spare"], d, generator=gen, device="cuda").to(DTYPES[case["dtype"]])
        axes = len(case["sections"].split(","))
        top = torch.tensor([120.0, 64.0, 64.0, 1000.0][:axes], device="cuda")
        pos = torch.floor(torch.rand(b, t, axes, generator=gen, device="cuda") * top)
        if case["pos"] == "f32":
            pos = pos * 0.375  # resampled frames and grids
        return case, buf[:, :, :h], pos.to(POS[case["pos"]])
    r, c, g = case["rows"], case["cols"], case["groups"]
    dt = DTYPES[case["dtype"]]
    pt = dt if case["pdtype"] == "same" else DTYPES[case["pdtype"]]
    x = (_activations(gen, r, c, torch.float32) + 0.25).to(dt)
    gain = bias = None
    if case["affine"] != "none":
        shift = 0.0 if case["affine"] == "modulate" else 1.0
        gain = (shift + 0.1 * torch.randn(g, c, generator=gen, device="cuda")).to(pt)
        bias = (0.1 * torch.randn(g, c, generator=gen, device="cuda")).to(pt)
    if op == "ln_forward":
        return case, x, gain, bias
    dy = torch.randn(r, c, generator=gen, device="cuda").to(dt)
    x32 = x.float()
    mean = x32.mean(1)
    rstd = torch.rsqrt((x32 - mean[:, None]).square().mean(1) + 1e-6)
    return case, dy, x, mean, rstd, gain


# --------------------------------------------------------------- one pass
def run(state):
    case = state[0]
    return _run_own(case, state[1:]) if own else globals()["_plain_" + case["op"]](case, *state[1:])


def _run_own(case, s):
    import diffusion_transformer_image_nvfp4_b200 as kl

    op = case["op"]
    if op == "quantize":
        q = kl.quantize_fp8_block(s[0], block=case["block"], transpose=case["transpose"], layout=case["layout"])
        return q.codes.view(torch.float8_e4m3fn), q.scales.view(torch.float8_e8m0fnu)
    if op == "gemm":
        a = kl.FP8Block(s[0], s[1], case["m"], case["k"])
        w = kl.FP8Block(s[2], s[3], case["n"], case["k"])
        return kl.gemm_fp8_block(a, w, out_dtype=DTYPES[case["out"]])
    if op == "rope":
        return kl.rope_axes(s[0], s[1], [int(n) for n in case["sections"].split(",")], theta=10000.0,
                            pairing=case["pairing"], ladder=case["ladder"], inverse=case["inverse"])
    if op == "ln_forward":
        return kl.layer_norm_forward(s[0], s[1], s[2], modulate=case["affine"] == "modulate", eps=1e-6)
    return kl.layer_norm_backward(s[0], s[1], s[2], s[3], s[4], modulate=case["affine"] == "modulate",
                                  groups=case["groups"])


def _plain_quantize(case, x):
    x = x.float()
    codes, s = _encode(x.t() if case["transpose"] else x, case["block"])
    if case["layout"] == "mma":
        s = _mma_scales(s)
    elif case["block"] == "tile":
        s = s[::128].contiguous()
    return codes.view(torch.float8_e4m3fn), s.view(torch.float8_e8m0fnu)


def _decode(codes, scales, rows, cols):
    s = _linear_scales(scales, rows, cols).int() - 127
    v = codes.view(torch.float8_e4m3fn)[:, :cols].float()
    return v * _pow2(s).repeat_interleave(128, 1)[:, :cols]


def _plain_gemm(case, a, sa, w, sw):
    m, n, k = case["m"], case["n"], case["k"]
    return (_decode(a, sa, m, k) @ _decode(w, sw, n, k).t()).to(DTYPES[case["out"]])


def _plain_rope(case, x, pos):
    sections = torch.tensor([int(n) for n in case["sections"].split(",")], device=x.device)
    pairs = int(sum(int(n) for n in case["sections"].split(",")))
    j = torch.arange(pairs, device=x.device, dtype=torch.float64)
    axis = torch.arange(len(sections), device=x.device).repeat_interleave(sections, output_size=pairs)
    n = sections[axis].double()
    u = j - (sections.cumsum(0) - sections)[axis].double()
    expo = u / n if case["ladder"] == "axis" else j / pairs
    ang = pos.double()[:, :, axis] * torch.exp(-math.log(10000.0) * expo)  # 64 bits: far positions
    if case["inverse"]:
        ang = -ang
    c, s = ang.cos().float()[:, :, None], ang.sin().float()[:, :, None]
    v = x.float()
    rot = v[..., :2 * pairs]
    if case["pairing"] == "half":
        a, b = rot[..., :pairs], rot[..., pairs:]
        new = torch.cat([a * c - b * s, a * s + b * c], -1)
    else:
        a, b = rot[..., 0::2], rot[..., 1::2]
        new = torch.stack([a * c - b * s, a * s + b * c], -1).flatten(-2)
    return torch.cat([new, v[..., 2 * pairs:]], -1).to(x.dtype)


def _grouped(p, rows):
    return p.float().repeat_interleave(rows // p.shape[0], 0)


def _plain_ln_forward(case, x, gain, bias):
    v = x.float()
    mean = v.mean(1, keepdim=True)
    d = v - mean
    rstd = torch.rsqrt(d.square().mean(1, keepdim=True) + 1e-6)
    y = d * rstd
    if gain is not None:
        g = _grouped(gain, len(v))
        y = y * (1.0 + g if case["affine"] == "modulate" else g) + _grouped(bias, len(v))
    return y.to(x.dtype), mean[:, 0], rstd[:, 0]


def _plain_ln_backward(case, dy, x, mean, rstd, gain):
    d = dy.float()
    xhat = (x.float() - mean[:, None]) * rstd[:, None]
    h = d
    if gain is not None:
        g = _grouped(gain, len(d))
        h = d * (1.0 + g if case["affine"] == "modulate" else g)
    dx = rstd[:, None] * (h - h.mean(1, keepdim=True) - xhat * (h * xhat).mean(1, keepdim=True))
    groups = case["groups"]
    dgain = (d * xhat).view(groups, -1, d.shape[1]).sum(1)
    dbias = d.view(groups, -1, d.shape[1]).sum(1)
    return dx.to(x.dtype), dgain, dbias


# ------------------------------------------------- the definitions, 64 bits
def exact(case, seed):
    s = prepare(case, seed)[1:]
    op = case["op"]
    if op == "quantize":
        return _exact_quantize(case, s[0].double())
    if op == "gemm":
        a, w = (_exact_decode(c, b, r, case["k"]) for c, b, r in ((s[0], s[1], case["m"]), (s[2], s[3], case["n"])))
        return torch.einsum("mk,nk->mn", a, w)
    if op == "rope":
        return _exact_rope(case, s[0].double(), s[1].double())
    if op == "ln_forward":
        return _exact_ln_forward(case, *s)
    return _exact_ln_backward(case, *s)


def _exact_quantize(case, x):
    if case["transpose"]:
        x = x.t().contiguous()
    r, c = x.shape
    rb, cb = -(-r // 128), -(-c // 128)
    p = torch.nn.functional.pad(x, (0, cb * 128 - c, 0, rb * 128 - r)).reshape(rb, 128, cb, 128)
    top = p.abs().amax(3) if case["block"] == "row" else p.abs().amax((1, 3))[:, None].expand(rb, 128, cb)
    # the margin is far below the step between 32-bit values: it keeps an exact power of two from rounding up
    e = torch.ceil(torch.log2(top / 448.0) - 1e-9).clamp(-127, 127)
    scale = torch.where(top == 0, torch.ones_like(top), torch.exp2(e))
    v = p / scale[..., None]
    step = torch.exp2(torch.floor(torch.log2(v.abs())).clamp(min=-6) - 3)
    codes = (torch.round(v / step) * step).reshape(rb * 128, cb * 128)
    codes = codes[:r, :-(-c // 16) * 16]
    if case["layout"] == "linear":
        flat = scale.reshape(rb * 128, cb)[:r] if case["block"] == "row" else scale[:, 0]
        return codes, flat
    ab = -(-cb // 4)
    atoms = torch.full((rb, ab, 32, 4, 4), 2.0 ** -127, dtype=torch.float64, device=x.device)
    row, blk = torch.meshgrid(torch.arange(r, device=x.device), torch.arange(cb, device=x.device), indexing="ij")
    atoms[row // 128, blk // 4, row % 32, row % 128 // 32, blk % 4] = scale.reshape(rb * 128, cb)[:r]
    return codes, atoms.flatten()


def _exact_decode(codes, flat, rows, cols):
    table = torch.arange(256, dtype=torch.uint8, device=codes.device).view(torch.float8_e4m3fn).double()
    row, col = torch.arange(rows, device=codes.device)[:, None], torch.arange(0, cols, 128, device=codes.device) // 128
    per_row = 512 * (-(-len(col) // 4))
    at = row // 128 * per_row + col // 4 * 512 + row % 32 * 16 + row % 128 // 32 * 4 + col % 4
    scale = torch.exp2(flat[at].double() - 127.0)
    return table[codes[:, :cols].int()] * scale[:, torch.arange(cols, device=codes.device) // 128]


def _exact_rope(case, x, pos):
    parts, first, sections = [], 0, [int(n) for n in case["sections"].split(",")]
    for a, n in enumerate(sections):
        u = torch.arange(n, device=x.device, dtype=torch.float64)
        f = 10000.0 ** (-u / n if case["ladder"] == "axis" else -(first + u) / sum(sections))
        parts.append(pos[:, :, a, None] * f)
        first += n
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=x.device), torch.cat(parts, -1))[:, :, None]
    turn = turn.conj() if case["inverse"] else turn
    if case["pairing"] == "half":
        z = torch.complex(x[..., :first], x[..., first:2 * first]) * turn
        head = torch.cat([z.real, z.imag], -1)
    else:
        z = torch.view_as_complex(x[..., :2 * first].reshape(*x.shape[:-1], first, 2)) * turn
        head = torch.view_as_real(z).flatten(-2)
    return torch.cat([head, x[..., 2 * first:]], -1)


def _exact_ln_forward(case, x, gain, bias):
    x = x.double().view(case["groups"], -1, x.shape[1])
    var, mean = torch.var_mean(x, 2, correction=0, keepdim=True)
    rstd = (var + 1e-6) ** -0.5
    y = (x - mean) * rstd
    if gain is not None:
        y = y * (gain.double() + (case["affine"] == "modulate"))[:, None] + bias.double()[:, None]
    return y.flatten(0, 1), mean.flatten(), rstd.flatten()


def _exact_ln_backward(case, dy, x, mean, rstd, gain):
    shape = (case["groups"], -1, x.shape[1])
    dy, x = dy.double().view(shape), x.double().view(shape)
    r = rstd.double().view(case["groups"], -1, 1)
    xhat = (x - mean.double().view(case["groups"], -1, 1)) * r
    h = dy if gain is None else dy * (gain.double() + (case["affine"] == "modulate"))[:, None]
    along = torch.einsum("grc,grc->gr", h, xhat)[..., None] / x.shape[2]
    dx = (h - h.sum(2, keepdim=True) / x.shape[2] - xhat * along) * r
    return dx.flatten(0, 1), torch.einsum("grc,grc->gc", dy, xhat), dy.sum(1)
