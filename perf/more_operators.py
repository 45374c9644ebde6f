"""The operators of a low-precision linear layer, as they are timed: root-mean-square norm with the residual's addition
(forward, with 8-bit output, and backward), 4-bit microscaled packing, and the product of 4-bit weights with 4-bit or
8-bit rows.

Each case is one call (for packing: the pair of calls that stores and restores). `run` computes it from elementary torch
operations, or, where `own` is true, by this package's kernels.

Held in 4 bits: per row and block of 32 columns, e2m1 values (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives) and one
power of two 2^e, e the least exponent (-126 .. 125) for which amax / 2^e rounds to at most 6; the scale byte is
e + 127, two values share a byte (the even column the lower half), rows are padded to whole blocks of 128 with zeros.
The scale bytes lie as [columns / 128, rows, 4].

Held in 8 bits: per row and block of 128 columns, e4m3 values and one power of two 2^e, e the least exponent
(-117 .. 120) with amax <= 448 * 2^e; the scale byte is e + 127.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
# bytes of a stored value, scales included
BYTES = {"bf16": 2, "f32": 4, "8": 1 + 1 / 128, "4": 0.5 + 1 / 32}


# ------------------------------------------------------------------------------------------------
# cases
# ------------------------------------------------------------------------------------------------
def listed():
    return [
        # one token of a generation loop in the 12-layer d=1024 set: latency only
        dict(name="rms norm, 1x1024", op="norm", rows=1, cols=1024, x="bf16", residual="bf16", out="bf16"),
        # a training step's norm in the 24-layer d=2048 set: the branch is added to the stream, the linear layers read 8 bits
        dict(name="rms norm to 8 bits, 24576x2048", op="norm", rows=24576, cols=2048, x="bf16", residual="bf16", out="8"),
        # ragged rows, a fp32 stream beside a bf16 branch
        dict(name="rms norm, 1537x2047, f32 stream", op="norm", rows=1537, cols=2047, x="bf16", residual="f32", out="bf16"),
        # a training step's norm backwards, 12-layer d=1024 set, with the stream's own gradient
        dict(name="rms norm grad, 49152x1024", op="norm_grad", rows=49152, cols=1024, x="bf16", dy="bf16", stream=True),
        # a short ragged batch in fp32
        dict(name="rms norm grad, 129x1003 f32", op="norm_grad", rows=129, cols=1003, x="f32", dy="f32", stream=False),
        # a ragged gradient, packed along its tokens
        dict(name="4 bits, 1003x333 f32, transposed", op="pack", rows=1003, cols=333, x="f32", out="f32", transpose=True),
        # c_fc's weights of the 32-layer d=4096 set, after an optimizer step
        dict(name="4 bits, 16384x4096 bf16", op="pack", rows=16384, cols=4096, x="bf16", out="bf16", transpose=False),
        # one token through c_fc of the 32-layer d=4096 set
        dict(name="product, 1 x (16384x4096)", op="product", rows=1, outs=16384, ins=4096, x="8", out="bf16", accumulate=False),
        # ragged everything, added to what is there
        dict(name="product, 129 x (1003x333) f32", op="product", rows=129, outs=1003, ins=333, x="4", out="f32", accumulate=True),
        # a projection back into the fp32 stream, 24-layer d=2048 set
        dict(name="product, 24576 x (2048x8192)", op="product", rows=24576, outs=2048, ins=8192, x="4", out="f32", accumulate=True),
        # c_fc of the 32-layer d=4096 set
        dict(name="product, 12288 x (16384x4096)", op="product", rows=12288, outs=16384, ins=4096, x="4", out="bf16", accumulate=False),
        # its c_proj, rows in 8 bits
        dict(name="product of 8 bits, 12288 x (4096x16384)", op="product", rows=12288, outs=4096, ins=16384, x="8", out="bf16", accumulate=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _size(rng, lo, hi, step):
    """Spread over the logarithm; two in three at a multiple of `step` (as models have them), the rest anywhere."""
    n = _log(rng, lo, hi)
    return max(step, n // step * step) if rng.random() < 0.67 else n


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "pack", "product", "product"])
    t = lambda: rng.choice(["bf16", "f32"])  # noqa: E731
    if op == "product":
        c = dict(op=op, rows=_log(rng, 1, 24576), outs=_size(rng, 16, 16384, 64), ins=_size(rng, 16, 16384, 64), x=rng.choice(["4", "8"]), out=t(), accumulate=rng.random() < 0.3)
        while c["rows"] * c["outs"] * c["ins"] > 12288 * 16384 * 4096:
            c["rows"] = c["rows"] // 2
        return c
    c = dict(op=op, rows=_log(rng, 1, 32768), cols=_size(rng, 16, 8192 if op == "pack" else 4096, 64))
    if op == "norm":
        return dict(c, x=t(), residual=rng.choice(["bf16", "f32", "none"]), out=rng.choice(["bf16", "f32", "8"]))
    if op == "norm_grad":
        return dict(c, x=rng.choice(["bf16", "f32", "8"]), dy=t(), stream=rng.random() < 0.6)
    return dict(c, x=t(), out=t(), transpose=rng.random() < 0.5)


def work(case):
    c = case
    if c["op"] == "product":
        m, n, k = c["rows"], c["outs"], c["ins"]
        return {"bytes": m * k * BYTES[c["x"]] + n * k * BYTES["4"] + m * n * BYTES[c["out"]] * (2 if c["accumulate"] else 1), "flops": 2 * m * n * k}
    r, k = c["rows"], c["cols"]
    if c["op"] == "norm":
        # the residual is read and their sum written; 8 bits are written, and their values come back as bf16
        b = r * k * (BYTES[c["x"]] + BYTES[c["out"]]) + r * 4 + 4 * k
        b += 0 if c["residual"] == "none" else 2 * r * k * BYTES[c["residual"]]
        return {"bytes": b + (r * k * 2 if c["out"] == "8" else 0), "flops": 5 * r * k}
    if c["op"] == "norm_grad":
        dx = BYTES[c["dy"] if c["x"] == "8" else c["x"]]
        return {"bytes": r * k * (BYTES[c["x"]] + BYTES[c["dy"]] + dx * (2 if c["stream"] else 1)) + r * 4 + 8 * k, "flops": 11 * r * k}
    return {"bytes": r * k * (BYTES[c["x"]] + BYTES["4"] + BYTES[c["out"]]), "flops": 4 * r * k}


# ------------------------------------------------------------------------------------------------
# the two formats, in plain form
# ------------------------------------------------------------------------------------------------
def _blocks(x, block):
    """x in fp32 as [rows, blocks, block], padded with zeros to whole blocks of 128 columns."""
    rows, cols = x.shape
    return torch.nn.functional.pad(x.float(), (0, -cols % 128)).view(rows, -1, block)


def _pack8(x):
    """e4m3 bytes and scale bytes of x."""
    v = _blocks(x, 128)
    finite = v.isfinite()
    m, e = torch.frexp(torch.where(finite, v.abs(), torch.zeros_like(v)).amax(-1))
    e = torch.where(m > 0, e - 9 + (m > 0.875), torch.full_like(e, -117)).clamp(-117, 120)
    most = torch.where(e == 120, 240.0, 448.0)[..., None]
    q = torch.ldexp(v, -e[..., None])
    q = torch.where(finite, torch.minimum(torch.maximum(q, -most), most), float("nan")).to(torch.float8_e4m3fn)
    return q.view(x.shape[0], -1).view(torch.uint8), (e + 127).to(torch.uint8)


def _unpack8(q, scale, cols):
    s = torch.ldexp(torch.ones_like(scale, dtype=torch.float32), scale.int() - 127)
    return (q.view(torch.float8_e4m3fn).float().view(*scale.shape, 128) * s[..., None]).view(q.shape[0], -1)[:, :cols]


def _pack4(x):
    """Bytes of two e2m1 values each and scale bytes of x."""
    v = _blocks(x, 32)
    amax = v.abs().amax(-1)
    m, e = torch.frexp(amax)                                  # amax = m 2^e, m in [0.5, 1)
    e = torch.where(amax > 0, e - 3 + (m >= 0.875), torch.full_like(e, -126)).clamp(-126, 125)
    a = torch.ldexp(v.abs(), -e[..., None])
    # how many halfway points lie below; at one, the even neighbour
    code = (a > 0.25).byte() + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5)
    code = (code + 8 * torch.signbit(v)).to(torch.uint8).view(x.shape[0], -1)
    bad = ~amax.isfinite()
    code = torch.where(bad.repeat_interleave(32, 1), 0, code).to(torch.uint8)
    scale = torch.where(bad, 255, e + 127).to(torch.uint8)
    return code[:, ::2] | code[:, 1::2] << 4, scale.view(x.shape[0], -1, 4).transpose(0, 1).contiguous()


def _unpack4(q, scale, cols):
    values = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], device=q.device)
    scale = scale.transpose(0, 1).reshape(q.shape[0], -1)
    v = values[torch.stack([q & 15, q >> 4], -1).long()].view(*scale.shape, 32)
    s = torch.ldexp(torch.ones_like(scale, dtype=torch.float32), scale.int() - 127)
    s = torch.where(scale == 255, float("nan"), s)
    return (v * s[..., None]).view(q.shape[0], -1)[:, :cols]


# ------------------------------------------------------------------------------------------------
# inputs
# ------------------------------------------------------------------------------------------------
def _activations(g, rows, cols, dtype):
    """Residual-stream values: unit spread, an offset and a scale for each feature, a few large features."""
    x = torch.randn(rows, cols, generator=g, device="cuda")
    f = torch.rand(cols, generator=g, device="cuda")
    return (x * torch.where(f > 0.99, 20.0, 0.5 + f) + torch.randn(cols, generator=g, device="cuda") * 0.3).to(dtype)


def prepare(case, seed):
    c, g = case, torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = dict(c, case=c)
    if c["op"] == "product":
        x = _activations(g, c["rows"], c["ins"], torch.bfloat16)
        s["xq"], s["xs"] = _pack4(x) if c["x"] == "4" else _pack8(x)
        s["wq"], s["ws"] = _pack4(torch.randn(c["outs"], c["ins"], generator=g, device="cuda") * 0.02)
        if c["accumulate"]:
            s["y"] = _activations(g, c["rows"], c["outs"], DTYPES[c["out"]])
        return s
    x = _activations(g, c["rows"], c["cols"], DTYPES.get(c["x"], torch.bfloat16))
    if c["op"] == "pack":
        s["x"] = x
        return s
    s["gain"] = 1 + 0.2 * torch.randn(c["cols"], generator=g, device="cuda")
    if c["op"] == "norm":
        s["x"] = x
        s["stream"] = None if c["residual"] == "none" else 2 * torch.randn(c["rows"], c["cols"], generator=g, device="cuda").to(DTYPES[c["residual"]])
        return s
    s["rstd"] = (x.double().square().mean(1) + 1e-5).rsqrt().float()
    s["dy"] = (torch.randn(c["rows"], c["cols"], generator=g, device="cuda") * 1e-2).to(DTYPES[c["dy"]])
    kind = s["dy"].dtype if c["x"] == "8" else x.dtype
    s["dstream"] = (torch.randn(c["rows"], c["cols"], generator=g, device="cuda") * 1e-2).to(kind) if c["stream"] else None
    if c["x"] == "8":
        s["q"], s["scale"] = _pack8(x)
    else:
        s["x"] = x
    return s


# ------------------------------------------------------------------------------------------------
# one pass
# ------------------------------------------------------------------------------------------------
def _norm(s):
    if own:
        import adamw_optimizer_step_amd as ma
        x = s["x"]
        if s["out"] != "8":
            return list(ma.rmsnorm_forward(x, s["gain"], s["stream"], eps=1e-5, dtype=DTYPES[s["out"]]))
        held = ma.ActCheckpoint.empty(*x.shape, device=x.device)
        _, total, rstd = ma.rmsnorm_forward(x, s["gain"], s["stream"], eps=1e-5, held=held)
        return [ma.act_unpack(held, dtype=torch.bfloat16), total, rstd]
    total = s["x"] if s["stream"] is None else (s["x"].float() + s["stream"].float()).to(s["stream"].dtype)
    h = total.float()
    rstd = torch.rsqrt((h * h).mean(1) + 1e-5)
    y = h * rstd[:, None] * s["gain"]
    y = _unpack8(*_pack8(y), s["cols"]).bfloat16() if s["out"] == "8" else y.to(DTYPES[s["out"]])
    return [y, total, rstd]


def _norm_grad(s):
    if own:
        import adamw_optimizer_step_amd as ma
        x = ma.ActCheckpoint(s["q"], s["scale"], s["cols"]) if s["case"]["x"] == "8" else s["x"]
        dgain = torch.empty_like(s["gain"])
        return [ma.rmsnorm_backward(s["dy"], x, s["rstd"], s["gain"], dtotal=s["dstream"], dgain=dgain), dgain]
    x = _unpack8(s["q"], s["scale"], s["cols"]) if s["case"]["x"] == "8" else s["x"].float()
    dy, rstd = s["dy"].float(), s["rstd"][:, None]
    xh, g = x * rstd, dy * s["gain"]
    dx = rstd * (g - xh * (g * xh).mean(1, keepdim=True))
    if s["dstream"] is not None:
        dx = dx + s["dstream"].float()
    return [dx.to(s["dy"].dtype if s["case"]["x"] == "8" else s["x"].dtype), (dy * xh).sum(0)]


def _pack(s):
    if own:
        import adamw_optimizer_step_amd as ma
        return ma.mx4_unpack(ma.mx4_pack(s["x"], transpose=s["transpose"]), dtype=DTYPES[s["out"]])
    x = s["x"].t() if s["transpose"] else s["x"]
    return _unpack4(*_pack4(x), x.shape[1]).to(DTYPES[s["out"]])


def _product(s):
    if own:
        import adamw_optimizer_step_amd as ma
        x = (ma.Mx4Matrix if s["x"] == "4" else ma.ActCheckpoint)(s["xq"], s["xs"], s["ins"])
        w = ma.Mx4Matrix(s["wq"], s["ws"], s["ins"])
        if s["accumulate"]:
            return ma.mx4_matmul(x, w, out=s["y"], accumulate=True)
        return ma.mx4_matmul(x, w, dtype=DTYPES[s["out"]])
    x = (_unpack4 if s["x"] == "4" else _unpack8)(s["xq"], s["xs"], s["ins"])
    y = x @ _unpack4(s["wq"], s["ws"], s["ins"]).t()
    if s["accumulate"]:
        return s["y"].copy_(s["y"].float() + y)
    return y.to(DTYPES[s["out"]])


OPS = {"norm": _norm, "norm_grad": _norm_grad, "pack": _pack, "product": _product}


def run(state):
    return OPS[state["op"]](state)


# ------------------------------------------------------------------------------------------------
# the definition, in 64 bits
# ------------------------------------------------------------------------------------------------
def _nearest(v, mantissa, least):
    """The nearest number of `mantissa` bits after the leading one to each v, ties to even; steps of `least` at least."""
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=1e-300))) - mantissa).clamp(min=least)
    return torch.round(v / step) * step


def _held8(x):
    rows, cols = x.shape
    v = torch.nn.functional.pad(x.double(), (0, -cols % 128)).view(rows, -1, 128)
    amax = v.abs().amax(-1, keepdim=True)
    e = torch.ceil(torch.log2(amax.clamp(min=1e-300) / 448)).clamp(-117, 120)
    e = e + (amax > 448 * torch.exp2(e)).double() - ((amax <= 448 * torch.exp2(e - 1)) & (e > -117)).double()
    return (_nearest(v / torch.exp2(e), 3, 2.0 ** -9) * torch.exp2(e)).view(rows, -1)[:, :cols]


def _held4(x):
    rows, cols = x.shape
    v = torch.nn.functional.pad(x.double(), (0, -cols % 32)).view(rows, -1, 32)
    most = _nearest(v.abs().amax(-1, keepdim=True), 1, 2.0 ** -127)   # 1 or 1.5 times a power of two, or 0
    e = torch.ceil(torch.log2(most.clamp(min=1e-300) / 6)).clamp(-126, 125)
    return (_nearest(v / torch.exp2(e), 1, 0.5) * torch.exp2(e)).view(rows, -1)[:, :cols]


def _value8(q, scale, cols):
    """sign, 4 bits of exponent with bias 7, 3 of fraction"""
    q = q.long()
    e, f = (q >> 3) & 15, (q & 7).double()
    v = torch.where(e > 0, (8 + f) * torch.exp2(e.double() - 10), f * 2.0 ** -9)
    return (torch.where(q >= 128, -v, v) * torch.exp2(scale.double() - 127).repeat_interleave(128, 1))[:, :cols]


def _value4(q, scale, cols):
    """sign, 2 bits of exponent with bias 1, 1 of fraction"""
    scale = scale.permute(1, 0, 2).flatten(1)
    q = torch.stack([q % 16, q // 16], 2).flatten(1).long()
    e, f = (q % 8) // 2, (q % 2).double()
    v = torch.where(e > 0, (2 + f) * torch.exp2(e.double() - 2), f / 2)
    return (torch.where(q >= 8, -v, v) * torch.exp2(scale.double() - 127).repeat_interleave(32, 1))[:, :cols]


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "pack":
        return _held4(s["x"].t() if c["transpose"] else s["x"])
    if c["op"] == "product":
        x = (_value4 if c["x"] == "4" else _value8)(s["xq"], s["xs"], c["ins"])
        y = torch.mm(_value4(s["wq"], s["ws"], c["ins"]), x.t()).t()
        return y + s["y"].double() if c["accumulate"] else y
    gain = s["gain"].double()
    if c["op"] == "norm":
        h = s["x"].double()
        if s["stream"] is not None:
            h = (h + s["stream"].double()).to(s["stream"].dtype).double()   # the stream as it is stored
        rstd = ((h ** 2).sum(1) / c["cols"] + 1e-5) ** -0.5
        y = torch.einsum("ij,i,j->ij", h, rstd, gain)
        return [_held8(y) if c["out"] == "8" else y, h, rstd]
    x = _value8(s["q"], s["scale"], c["cols"]) if c["x"] == "8" else s["x"].double()
    dy, rstd, n = s["dy"].double(), s["rstd"].double(), c["cols"]
    g = dy * gain
    dx = rstd[:, None] * g - x * (rstd ** 3 * (g * x).sum(1) / n)[:, None]
    dx = dx if s["dstream"] is None else dx + s["dstream"].double()
    return [dx, torch.einsum("ij,ij,i->j", dy, x, rstd)]
