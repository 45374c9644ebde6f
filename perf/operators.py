"""The operators around the optimizer step, as they are timed: the embedding lookup and its gradient, layer norm
forward and backward, 8-bit activation checkpoints and the weight gradient that reads one.

Each case is one call (for a checkpoint: the pair of calls that stores and restores it). `run` computes it from
elementary torch operations, or, where `own` is true, by this package's kernels.

A checkpoint holds, per row and block of 128 columns, e4m3 values and one power of two 2^e, e the least exponent
(-117 .. 120) with amax <= 448 * 2^e; the scale byte is e + 127, rows are padded to whole blocks with zeros.
"""
import math

import torch

own = False

BLOCK = 128
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"bf16": 2, "f32": 4}


# ------------------------------------------------------------------------------------------------
# cases
# ------------------------------------------------------------------------------------------------
def listed():
    return [
        # one token of a generation loop, the 4-layer d=256 set's table: latency only
        dict(name="lookup, 1 token, 32768x256", op="lookup", rows=32768, cols=256, tokens=1, table="f32", out="f32", ignored=0.0),
        # a training step's lookup in the 12-layer d=1024 set's fp32 table, bf16 activations
        dict(name="lookup, 49152 tokens, 50304x1024", op="lookup", rows=50304, cols=1024, tokens=49152, table="f32", out="bf16", ignored=0.0),
        # a shard of a ragged table with ignored positions, added to a gradient that is already there
        dict(name="lookup grad, odd, accumulated", op="lookup_grad", rows=10007, cols=333, tokens=5003, dout="f32", ignored=0.25, accumulate=True),
        # the gradient AdamW reads for the 12-layer set's table, Zipf-distributed tokens
        dict(name="lookup grad, 49152 tokens, 50304x1024", op="lookup_grad", rows=50304, cols=1024, tokens=49152, dout="bf16", ignored=0.0, accumulate=False),
        # a few rows of fp32 activations: latency
        dict(name="norm, 8x256 f32", op="norm", rows=8, cols=256, x="f32", out="f32", affine=True, checkpoint=False),
        # a training step's norm that also leaves its input's checkpoint, 24-layer d=2048 set
        dict(name="norm + checkpoint, 24576x2048", op="norm", rows=24576, cols=2048, x="bf16", out="bf16", affine=True, checkpoint=True),
        # the backward of a training step's norm, 12-layer d=1024 set
        dict(name="norm grad, 49152x1024", op="norm_grad", rows=49152, cols=1024, x="bf16", dy="bf16", affine=True),
        # ragged rows out of a checkpoint, fp32 gradients
        dict(name="norm grad of checkpoint, 1537x2047", op="norm_grad", rows=1537, cols=2047, x="ckpt", dy="f32", affine=True),
        # a short ragged batch stored and restored
        dict(name="checkpoint, 129x1003 f32", op="checkpoint", rows=129, cols=1003, x="f32", out="f32"),
        # the MLP input of the 32-layer d=4096 set
        dict(name="checkpoint, 24576x4096 bf16", op="checkpoint", rows=24576, cols=4096, x="bf16", out="bf16"),
        # a ragged projection, fp32 gradients over micro-batches
        dict(name="weight grad, 1000x(250x333) f32", op="weight_grad", tokens=1000, outs=250, ins=333, dy="f32", grad="f32", accumulate=True),
        # c_fc's gradient of the 32-layer d=4096 set, what its Muon group reads
        dict(name="weight grad, 12288x(16384x4096)", op="weight_grad", tokens=12288, outs=16384, ins=4096, dy="bf16", grad="bf16", accumulate=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _size(rng, lo, hi, step):
    """Spread over the logarithm; two in three at a multiple of `step` (as models have them), the rest anywhere."""
    n = _log(rng, lo, hi)
    return max(step, n // step * step) if rng.random() < 0.67 else n


def draw(rng):
    op = rng.choice(["lookup", "lookup_grad", "norm", "norm_grad", "checkpoint", "weight_grad"])
    t = lambda: rng.choice(["bf16", "f32"])  # noqa: E731
    if op in ("lookup", "lookup_grad"):
        c = dict(op=op, rows=_log(rng, 256, 65536), cols=_size(rng, 64, 2048, 64), tokens=_log(rng, 1, 65536), ignored=rng.choice([0.0, 0.0, round(rng.random(), 2)]))
        return {**c, "table": t(), "out": t()} if op == "lookup" else {**c, "dout": t(), "accumulate": rng.random() < 0.4}
    if op == "weight_grad":
        return dict(op=op, tokens=_log(rng, 1, 24576), outs=_size(rng, 16, 8192, 64), ins=_size(rng, 16, 4096, 64), dy=rng.choice(["bf16", "bf16", "f32"]), grad=t(), accumulate=rng.random() < 0.3)
    c = dict(op=op, rows=_log(rng, 1, 32768), cols=_size(rng, 16, 4096, 64))
    if op == "norm":
        return dict(c, x=t(), out=t(), affine=rng.random() < 0.8, checkpoint=rng.random() < 0.4)
    if op == "norm_grad":
        return dict(c, x=rng.choice(["bf16", "f32", "ckpt"]), dy=t(), affine=rng.random() < 0.8)
    return dict(c, x=t(), out=t())


def _distinct(rows, tokens):
    """How many different rows Zipf-distributed tokens touch (expected)."""
    i = torch.arange(rows, dtype=torch.float64)
    p = (torch.log(i + 2) - torch.log(i + 1)) / math.log(rows + 1)
    return float((-torch.expm1(tokens * torch.log1p(-p.clamp(max=1 - 1e-12)))).sum())


def work(case):
    c = case
    if c["op"] == "lookup":
        n = c["tokens"] * (1 - c["ignored"])
        return {"bytes": _distinct(c["rows"], n) * c["cols"] * BYTES[c["table"]] + c["tokens"] * (8 + c["cols"] * BYTES[c["out"]]), "flops": n * c["cols"]}
    if c["op"] == "lookup_grad":
        n = c["tokens"] * (1 - c["ignored"])
        grad = 2 * _distinct(c["rows"], n) if c["accumulate"] else c["rows"]
        return {"bytes": n * c["cols"] * BYTES[c["dout"]] + c["tokens"] * 8 + grad * c["cols"] * 4, "flops": n * c["cols"]}
    if c["op"] == "weight_grad":
        t, n, k = c["tokens"], c["outs"], c["ins"]
        return {"bytes": t * n * BYTES[c["dy"]] + t * k * (1 + 1 / BLOCK) + n * k * BYTES[c["grad"]] * (2 if c["accumulate"] else 1), "flops": 2 * t * n * k}
    r, k = c["rows"], c["cols"]
    held = 1 + 1 / BLOCK
    if c["op"] == "norm":
        b = r * k * (BYTES[c["x"]] + BYTES[c["out"]]) + r * 8 + (8 * k if c["affine"] else 0)
        # the checkpoint is written, and its values come back as bf16
        return {"bytes": b + (r * k * (held + 2) if c["checkpoint"] else 0), "flops": 8 * r * k}
    if c["op"] == "norm_grad":
        x = held if c["x"] == "ckpt" else BYTES[c["x"]]
        dx = BYTES[c["dy"] if c["x"] == "ckpt" else c["x"]]
        return {"bytes": r * k * (x + dx + BYTES[c["dy"]]) + r * 8 + (12 * k if c["affine"] else 0), "flops": 14 * r * k}
    return {"bytes": r * k * (BYTES[c["x"]] + held + BYTES[c["out"]]), "flops": 4 * r * k}


# ------------------------------------------------------------------------------------------------
# inputs
# ------------------------------------------------------------------------------------------------
def _tokens(g, rows, n, ignored):
    """Zipf-distributed ids; a share of the positions is ignored (an id outside the table)."""
    u = torch.rand(n, generator=g, device="cuda", dtype=torch.float64)
    t = (torch.exp(u * math.log(rows + 1)) - 1).long().clamp(0, rows - 1)
    return torch.where(torch.rand(n, generator=g, device="cuda") < ignored, torch.full_like(t, -1), t)


def _activations(g, rows, cols, dtype):
    """Residual-stream values: unit spread, an offset and a scale for each feature, a few large features."""
    x = torch.randn(rows, cols, generator=g, device="cuda")
    f = torch.rand(cols, generator=g, device="cuda")
    return (x * torch.where(f > 0.99, 20.0, 0.5 + f) + torch.randn(cols, generator=g, device="cuda") * 0.3).to(dtype)


def _pack(x):
    """Plain form of the checkpoint of x: e4m3 bytes and scale bytes."""
    rows, cols = x.shape
    blocks = -(-cols // BLOCK)
    v = torch.nn.functional.pad(x.float(), (0, blocks * BLOCK - cols)).view(rows, blocks, BLOCK)
    finite = v.isfinite()
    m, e = torch.frexp(torch.where(finite, v.abs(), torch.zeros_like(v)).amax(-1))
    e = torch.where(m > 0, e - 9 + (m > 0.875), torch.full_like(e, -117)).clamp(-117, 120)
    q = torch.ldexp(v, -e[..., None])
    most = torch.where(e == 120, 240.0, 448.0)[..., None]
    q = torch.where(finite, torch.minimum(torch.maximum(q, -most), most), float("nan")).to(torch.float8_e4m3fn)
    return q.view(rows, blocks * BLOCK).view(torch.uint8), (e + 127).to(torch.uint8)


def _unpack(q, scale, cols):
    """The values a checkpoint stands for, in fp32."""
    rows, blocks = scale.shape
    s = torch.ldexp(torch.ones_like(scale, dtype=torch.float32), scale.int() - 127)
    return (q.view(torch.float8_e4m3fn).float().view(rows, blocks, BLOCK) * s[..., None]).view(rows, -1)[:, :cols]


def prepare(case, seed):
    c, g = case, torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = dict(c, case=c)
    if c["op"] == "lookup":
        s["weight"] = (torch.randn(c["rows"], c["cols"], generator=g, device="cuda") * 0.02).to(DTYPES[c["table"]])
        s["ids"] = _tokens(g, c["rows"], c["tokens"], c["ignored"])
        s["by"] = math.sqrt(c["cols"])
    elif c["op"] == "lookup_grad":
        s["dy"] = (torch.randn(c["tokens"], c["cols"], generator=g, device="cuda") * 1e-3).to(DTYPES[c["dout"]])
        s["ids"] = _tokens(g, c["rows"], c["tokens"], c["ignored"])
        s["grad"] = torch.randn(c["rows"], c["cols"], generator=g, device="cuda") * 1e-3
        s["by"] = math.sqrt(c["cols"])
    elif c["op"] == "weight_grad":
        s["dy"] = (torch.randn(c["tokens"], c["outs"], generator=g, device="cuda") * 1e-3).to(DTYPES[c["dy"]])
        s["q"], s["scale"] = _pack(_activations(g, c["tokens"], c["ins"], torch.bfloat16))
        s["grad"] = (torch.randn(c["outs"], c["ins"], generator=g, device="cuda") * 1e-2).to(DTYPES[c["grad"]])
    else:
        x = _activations(g, c["rows"], c["cols"], DTYPES.get(c["x"], torch.bfloat16))
        if c["op"] != "checkpoint":
            s["gain"] = 1 + 0.2 * torch.randn(c["cols"], generator=g, device="cuda") if c["affine"] else None
            s["bias"] = 0.1 * torch.randn(c["cols"], generator=g, device="cuda") if c["affine"] else None
        if c["op"] == "norm_grad":
            f = x.double()
            var, mean = torch.var_mean(f, dim=1, correction=0)
            s["stats"] = torch.stack([mean, 1 / torch.sqrt(var + 1e-5)], 1).float().contiguous()
            s["dy"] = (torch.randn(c["rows"], c["cols"], generator=g, device="cuda") * 1e-2).to(DTYPES[c["dy"]])
            if c["x"] == "ckpt":
                s["q"], s["scale"] = _pack(x)
                return s
        s["x"] = x
    return s


# ------------------------------------------------------------------------------------------------
# one pass
# ------------------------------------------------------------------------------------------------
def _lookup(s):
    if own:
        import adamw_optimizer_step_amd as ma
        return ma.embedding_forward(s["weight"], s["ids"], scale=s["by"], dtype=DTYPES[s["out"]])
    ids = s["ids"]
    inside = (ids >= 0) & (ids < s["rows"])
    y = s["weight"][ids.clamp(0, s["rows"] - 1)].float() * s["by"]
    return torch.where(inside[:, None], y, 0.0).to(DTYPES[s["out"]])


def _lookup_grad(s):
    if own:
        import adamw_optimizer_step_amd as ma
        return ma.embedding_backward(s["dy"], s["ids"], s["grad"], scale=s["by"], accumulate=s["accumulate"])
    ids, grad = s["ids"], s["grad"]
    inside = (ids >= 0) & (ids < s["rows"])
    if not s["accumulate"]:
        grad.zero_()
    return grad.index_add_(0, ids.clamp(0, s["rows"] - 1), torch.where(inside[:, None], s["dy"].float() * s["by"], 0.0))


def _norm(s):
    if own:
        import adamw_optimizer_step_amd as ma
        x = s["x"]
        kept = ma.ActCheckpoint.empty(*x.shape, device=x.device) if s["checkpoint"] else None
        y, stats = ma.layernorm_forward(x, s["gain"], s["bias"], eps=1e-5, dtype=DTYPES[s["out"]], checkpoint=kept)
        return [y, stats] + ([ma.act_unpack(kept, dtype=torch.bfloat16)] if kept is not None else [])
    x = s["x"].float()
    mean = x.mean(1, keepdim=True)
    d = x - mean
    rstd = torch.rsqrt((d * d).mean(1, keepdim=True) + 1e-5)
    y = d * rstd
    if s["affine"]:
        y = y * s["gain"] + s["bias"]
    out = [y.to(DTYPES[s["out"]]), torch.cat([mean, rstd], 1)]
    return out + ([_unpack(*_pack(s["x"]), s["cols"]).bfloat16()] if s["checkpoint"] else [])


def _norm_grad(s):
    if own:
        import adamw_optimizer_step_amd as ma
        x = ma.ActCheckpoint(s["q"], s["scale"], s["cols"]) if s["case"]["x"] == "ckpt" else s["x"]
        if not s["affine"]:
            return [ma.layernorm_backward(s["dy"], x, s["stats"])]
        dgain, dbias = torch.empty_like(s["gain"]), torch.empty_like(s["bias"])
        return [ma.layernorm_backward(s["dy"], x, s["stats"], s["gain"], dgain=dgain, dbias=dbias), dgain, dbias]
    x = _unpack(s["q"], s["scale"], s["cols"]) if s["case"]["x"] == "ckpt" else s["x"].float()
    dy = s["dy"].float()
    mean, rstd = s["stats"][:, :1], s["stats"][:, 1:]
    xh = (x - mean) * rstd
    g = dy * s["gain"] if s["affine"] else dy
    dx = rstd * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
    dx = dx.to(s["dy"].dtype if s["case"]["x"] == "ckpt" else s["x"].dtype)
    return [dx, (dy * xh).sum(0), dy.sum(0)] if s["affine"] else [dx]


def _checkpoint(s):
    if own:
        import adamw_optimizer_step_amd as ma
        return ma.act_unpack(ma.act_pack(s["x"]), dtype=DTYPES[s["out"]])
    return _unpack(*_pack(s["x"]), s["cols"]).to(DTYPES[s["out"]])


def _weight_grad(s):
    if own:
        import adamw_optimizer_step_amd as ma
        return ma.act_weight_grad(s["dy"], ma.ActCheckpoint(s["q"], s["scale"], s["ins"]), s["grad"], accumulate=s["accumulate"])
    w = s["dy"].float().t() @ _unpack(s["q"], s["scale"], s["ins"])
    if s["accumulate"]:
        w = s["grad"].float() + w
    return s["grad"].copy_(w)


OPS = {"lookup": _lookup, "lookup_grad": _lookup_grad, "norm": _norm, "norm_grad": _norm_grad, "checkpoint": _checkpoint, "weight_grad": _weight_grad}


def run(state):
    return OPS[state["op"]](state)


# ------------------------------------------------------------------------------------------------
# the definition, in 64 bits
# ------------------------------------------------------------------------------------------------
def _e4m3(v):
    """The nearest e4m3 value of each v (|v| <= 448), ties to even: steps of 2^-3 of the leading power of two, 2^-9 at least."""
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(v / step) * step


def _held(x):
    """What the checkpoint of x stands for, in fp64, from the definition."""
    rows, cols = x.shape
    blocks = -(-cols // BLOCK)
    v = torch.nn.functional.pad(x.double(), (0, blocks * BLOCK - cols)).view(rows, blocks, BLOCK)
    amax = v.abs().amax(-1, keepdim=True)
    e = torch.ceil(torch.log2(amax.clamp(min=1e-300) / 448)).clamp(-117, 120)
    e = e + (amax > 448 * torch.exp2(e)).double() - ((amax <= 448 * torch.exp2(e - 1)) & (e > -117)).double()
    return (_e4m3(v / torch.exp2(e)) * torch.exp2(e)).view(rows, -1)[:, :cols]


def _e4m3_value(q):
    """The value of each e4m3 byte: sign, 4 bits of exponent with bias 7, 3 of fraction."""
    q = q.long()
    e, f = (q >> 3) & 15, (q & 7).double()
    v = torch.where(e > 0, (8 + f) * torch.exp2(e.double() - 10), f * 2.0 ** -9)
    return torch.where(q >= 128, -v, v)


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "lookup":
        by, w = float(torch.tensor(s["by"], dtype=torch.float32)), torch.cat([s["weight"].double(), torch.zeros(1, c["cols"], dtype=torch.float64, device="cuda")])
        return w[torch.where(s["ids"] < 0, c["rows"], s["ids"])] * by
    if c["op"] == "lookup_grad":
        by = float(torch.tensor(s["by"], dtype=torch.float32))
        order = torch.argsort(s["ids"], stable=True)
        order = order[s["ids"][order] >= 0]
        out = s["grad"].double() if c["accumulate"] else torch.zeros(c["rows"], c["cols"], dtype=torch.float64, device="cuda")
        return out.index_add(0, s["ids"][order], s["dy"][order].double() * by)
    if c["op"] == "checkpoint":
        return _held(s["x"])
    if c["op"] == "norm":
        x = s["x"].double()
        var, mean = torch.var_mean(x, dim=1, correction=0)
        rstd = (var + 1e-5) ** -0.5
        y = (x - mean[:, None]) * rstd[:, None]
        y = torch.addcmul(s["bias"].double(), y, s["gain"].double()) if c["affine"] else y
        return [y, torch.stack([mean, rstd], 1)] + ([_held(s["x"])] if c["checkpoint"] else [])
    if "q" in s:
        scales = torch.exp2(s["scale"].double() - 127).repeat_interleave(BLOCK, 1)
        x = (_e4m3_value(s["q"]) * scales)[:, : c.get("cols", c.get("ins"))]
    else:
        x = s["x"].double()
    dy = s["dy"].double()
    if c["op"] == "weight_grad":
        w = torch.mm(x.t(), dy).t()
        return w + s["grad"].double() if c["accumulate"] else w
    mean, rstd = s["stats"].double().unbind(1)
    xh = (x - mean[:, None]) * rstd[:, None]
    g = dy * s["gain"].double() if c["affine"] else dy
    n = c["cols"]
    dx = (n * g - g.sum(1, keepdim=True) - xh * (g * xh).sum(1, keepdim=True)) * (rstd / n)[:, None]
    return [dx, torch.einsum("ij,ij->j", dy, xh), dy.sum(0)] if c["affine"] else [dx]
