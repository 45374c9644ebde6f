"""GPU parity of the operators around the step against the fp64 oracle
(oracle/train_ops.py): embedding, layer norm, 8-bit checkpoints, the weight
gradient, and a run of them that ends in an optimizer step.

Error bounds are per element and follow from the operations: u = 2^-24 is half
an fp32 step; a sum of n fp32 terms in any order is off by at most n u times the
sum of the magnitudes (to first order); a result rounded once to type t is off
by half a step more, eps(t) / 2 of its value."""
import ctypes as C

import numpy as np
import pytest
import torch

import adamw_optimizer_step_amd as ma
from adamw_optimizer_step_amd import _lib as L
from gpu_util import need_gpu, say, to_np
from oracle import train_ops as T

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
F32, BF16 = torch.float32, torch.bfloat16
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


def half(dtype):
    return torch.finfo(dtype).eps / 2


def f64(t):
    return to_np(t).astype(np.float64)


def close(got, want, tol, dtype=F32):
    """|got - want| <= tol + half a step of `dtype`, elementwise; NaN and infinities alike. A result near the
    type's smallest normal number may be off by half its smallest subnormal."""
    got, want = f64(got), np.asarray(want, np.float64)
    assert got.shape == want.shape
    fin = np.isfinite(want)
    assert np.array_equal(np.isnan(got), np.isnan(want))
    assert np.array_equal(got[~fin & ~np.isnan(want)], want[~fin & ~np.isnan(want)])
    tol = np.broadcast_to(tol, want.shape)
    bound = (tol * (1 + half(dtype)) + half(dtype) * np.abs(want) + torch.finfo(dtype).smallest_normal * half(dtype) * 2)[fin]
    err = np.abs(got - want)[fin]
    assert np.all(err <= bound), f"off by up to {np.max(err / np.maximum(bound, 1e-300)):.3g} times the bound"


def rand(shape, seed, dtype=F32, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(dtype).to(DEV)


def view(t, off):
    """The same values at an element offset into a larger buffer (unaligned rows), guarded on both sides."""
    buf = torch.full((t.numel() + 2 * off + 64,), 7, dtype=t.dtype, device=DEV)
    v = buf[off: off + t.numel()].view(t.shape)
    v.copy_(t)
    return buf, v


def guards(buf, n, off):
    return bool((buf[:off] == 7).all()) and bool((buf[off + n:] == 7).all())


# ---------------------------------------------------------------------------
# embedding
# ---------------------------------------------------------------------------
TOKENS = {
    "spread": lambda r, n, g: torch.randint(0, r, (n,), generator=g),
    "zipf": lambda r, n, g: (torch.exp(torch.rand(n, generator=g, dtype=torch.float64) * np.log(r + 1)) - 1).long().clamp(0, r - 1),
    "one": lambda r, n, g: torch.full((n,), r // 2),
    "outside": lambda r, n, g: torch.randint(-r, 2 * r, (n,), generator=g),
    "none": lambda r, n, g: torch.full((n,), -1),
    "far": lambda r, n, g: torch.randint(0, r, (n,), generator=g) + (torch.arange(n) % 3 == 0) * (1 << 40),
}


def tokens(kind, rows, n, seed, dtype=torch.int64):
    return TOKENS[kind](rows, n, torch.Generator().manual_seed(seed)).to(dtype)


@pytest.mark.parametrize("rows,cols,n,td,od,kind,off", [
    (1, 1, 1, F32, F32, "spread", 0), (7, 3, 5, F32, BF16, "outside", 1), (300, 8, 64, BF16, F32, "spread", 0),
    (50, 130, 33, BF16, BF16, "zipf", 3), (50, 256, 17, F32, F32, "outside", 0), (1000, 333, 129, F32, BF16, "none", 1),
    (64, 1024, 70, F32, BF16, "zipf", 0), (33, 2056, 9, BF16, BF16, "far", 0), (4, 4099, 6, F32, F32, "spread", 2),
])
@pytest.mark.parametrize("idt", [torch.int32, torch.int64])
def test_embedding_forward(rows, cols, n, td, od, kind, off, idt):
    if kind == "far" and idt == torch.int32:
        pytest.skip("beyond int32")
    say("embedding_forward", rows, cols, n, td, od, kind, off, idt)
    w, t = rand((rows, cols), 1, td), tokens(kind, rows, n, 2, idt)
    _, wv = view(w, off)
    ob, ov = view(torch.zeros(n, cols, dtype=od, device=DEV), off)
    ma.embedding_forward(wv, t.to(DEV), scale=1.7, out=ov)
    # one fp32 product, then one rounding to the output's type
    close(ov, T.embedding_forward(f64(w), t.numpy(), 1.7), U * np.abs(T.embedding_forward(f64(w), t.numpy(), 1.7)), od)
    assert guards(ob, n * cols, off)


def test_embedding_shapes_and_defaults():
    w, t = rand((20, 16), 3, BF16), torch.randint(0, 20, (2, 3), device=DEV)
    y = ma.embedding_forward(w, t)
    assert y.shape == (2, 3, 16) and y.dtype == BF16 and torch.equal(y, w[t])
    assert ma.embedding_forward(w, t[:0], dtype=F32).shape == (0, 3, 16)
    g = torch.full((20, 16), 3.0, device=DEV)
    assert ma.embedding_backward(y[:0], t[:0], g, accumulate=True) is g and bool((g == 3).all())
    ma.embedding_backward(y[:0], t[:0], g)
    assert not g.any()


@pytest.mark.parametrize("rows,cols,n,dd,kind,off", [
    (1, 1, 1, F32, "spread", 0), (5, 3, 64, F32, "outside", 1), (5, 8, 65, BF16, "one", 0), (300, 40, 64, BF16, "spread", 1),
    (257, 512, 200, F32, "zipf", 0), (1000, 333, 3000, F32, "zipf", 1), (97, 1030, 1500, BF16, "zipf", 0),
    (30, 64, 5000, BF16, "one", 0), (700, 2050, 513, F32, "outside", 0), (66000, 16, 4097, BF16, "zipf", 0),
    (200000, 5, 2500, F32, "spread", 0), (40, 24, 100, F32, "none", 0), (3, 16, 20000, F32, "spread", 0),
    (70, 520, 512, BF16, "one", 0), (70, 520, 513, BF16, "one", 0), (9, 33, 511, F32, "outside", 1), (9, 33, 700, F32, "none", 0),
    (1 << 18, 3, 600, F32, "zipf", 0), (513, 8, 17000, BF16, "zipf", 0),
    (70, 520, 1024, BF16, "one", 0), (70, 520, 1025, BF16, "one", 0), (700, 2050, 1025, F32, "outside", 0), (9, 33, 1023, F32, "outside", 1),
    (40, 1033, 900, F32, "zipf", 1), (9, 33, 1100, F32, "none", 0), (1 << 18, 3, 1300, F32, "zipf", 0), (3, 8, 300000, BF16, "zipf", 0),
])
@pytest.mark.parametrize("acc", [False, True])
def test_embedding_backward(rows, cols, n, dd, kind, off, acc):
    say("embedding_backward", rows, cols, n, dd, kind, off, acc)
    t, d = tokens(kind, rows, n, 4), rand((n, cols), 5, dd)
    g0 = rand((rows, cols), 6)
    want, mag, count = T.embedding_backward(f64(d), t.numpy(), rows, -0.3, f64(g0) if acc else None)
    gb, gv = view(g0, off)
    _, dv = view(d, off)
    ma.embedding_backward(dv, t.to(DEV), gv, scale=-0.3, accumulate=acc)
    # count terms (the pieces of a long run add at most one each), the scale, and the addition to what was there
    tol = (count[:, None] * (1 + 1 / 64) + 3) * U * mag + (U * (np.abs(f64(g0)) + mag) if acc else 0)
    close(gv, want, tol)
    assert guards(gb, rows * cols, off)
    if acc:   # rows without a token keep their bits
        assert torch.equal(gv[torch.from_numpy(count == 0).to(DEV)], g0[torch.from_numpy(count == 0).to(DEV)])
    again = gv.clone() if not acc else g0.clone()
    ma.embedding_backward(d, t.to(DEV).int(), again, scale=-0.3, accumulate=acc)
    assert torch.equal(again, gv)   # the same bits for the same inputs, whatever the token type and alignment


def test_embedding_gradient_of_ignored_rows_is_not_read():
    """dout rows of ignored tokens may hold anything."""
    t = torch.tensor([3, -1, 3, 99], device=DEV)
    d = rand((4, 24), 7)
    d[1], d[3] = float("nan"), float("inf")
    g = torch.empty(10, 24, device=DEV)
    ma.embedding_backward(d, t, g)
    want = torch.zeros(10, 24, device=DEV)
    want[3] = d[0] + d[2]
    assert torch.equal(g, want)


def test_embedding_backward_is_the_transpose_of_forward():
    """<forward(w), d> = <w, backward(d)>: the forward is linear, so this is its difference quotient exactly."""
    w, t, d = rand((50, 96), 8), tokens("outside", 50, 400, 9).to(DEV), rand((400, 96), 10)
    y = ma.embedding_forward(w, t, scale=0.7)
    g = ma.embedding_backward(d, t, torch.empty(50, 96, device=DEV), scale=0.7)
    a, b = (y.double() * d.double()).sum().item(), (w.double() * g.double()).sum().item()
    mags = (y.double().abs() * d.double().abs()).sum().item()
    assert abs(a - b) <= 450 * U * mags


# ---------------------------------------------------------------------------
# layer norm
# ---------------------------------------------------------------------------
DEPTH = 48   # additions one after the other in a row's sum: 16 per lane, 6 in the wave, 16 over the waves, spare


def norm_inputs(rows, cols, xd, seed):
    x = rand((rows, cols), seed, F32, 2.0) + rand((rows, 1), seed + 1, F32, 3.0)
    if rows > 2:
        x[1] = 5.0      # no variance at all
    return x.to(xd), 1 + rand((cols,), seed + 2, F32, 0.3), rand((cols,), seed + 3, F32, 0.3)


NORM_SHAPES = [(1, 1), (3, 2), (5, 7), (1, 256), (9, 511), (4, 512), (6, 513), (130, 1024), (3, 1025), (2, 2048), (5, 2047), (3, 4096),
               (2, 4097), (2, 8200), (3, 16384), (2, 16383), (1000, 40), (512, 100), (513, 700), (600, 2049), (513, 1290), (1024, 300), (1025, 700), (1100, 2049),
               (1027, 4093), (515, 8189), (1026, 8190), (2100, 130), (4200, 130), (4200, 530), (2100, 1100),
               (260, 8200)]


@pytest.mark.parametrize("rows,cols", NORM_SHAPES)
@pytest.mark.parametrize("xd,yd,affine,off", [(F32, F32, True, 0), (BF16, BF16, True, 1), (BF16, F32, False, 0), (F32, BF16, False, 3)])
def test_layernorm_forward(rows, cols, xd, yd, affine, off):
    say("layernorm_forward", rows, cols, xd, yd, affine, off)
    x, gain, bias = norm_inputs(rows, cols, xd, 20)
    gain, bias = (gain, bias) if affine else (None, None)
    xn = f64(x)
    y, mean, rstd = T.layernorm_forward(xn, None if gain is None else f64(gain), None if bias is None else f64(bias))
    _, xv = view(x, off)
    yb, yv = view(torch.zeros(rows, cols, dtype=yd, device=DEV), off)
    ck = ma.ActCheckpoint.empty(rows, cols, DEV)
    out, stats = ma.layernorm_forward(xv, gain, bias, out=yv, checkpoint=ck)
    mean_tol = (DEPTH + 2) * U * np.abs(xn).mean(1, keepdims=True)
    dev = np.abs(xn - mean)
    # the variance: each squared difference is off by u(|x| + |mean|) + the mean's error in its factor, the sum by depth u
    var_abs = (2 * dev * (U * dev + mean_tol) + mean_tol ** 2).mean(1, keepdims=True) + (DEPTH + 3) * U * (dev ** 2).mean(1, keepdims=True)
    rstd_rel = 0.5 * var_abs * rstd ** 2 + 4 * U
    close(stats[:, :1], mean, mean_tol)
    close(stats[:, 1:], rstd, rstd * (rstd_rel + rstd_rel ** 2))
    g = np.abs(f64(gain)) if affine else 1.0
    xh = dev * rstd
    tol = g * (rstd * (mean_tol + 2 * U * dev) + xh * (rstd_rel + rstd_rel ** 2 + 3 * U)) * (1 + 1e-3) + U * np.abs(y) + (U * np.abs(f64(bias)) if affine else 0)
    close(yv, y, tol, yd)
    assert guards(yb, rows * cols, off)
    q, s = T.act_pack(xn)
    assert np.array_equal(ck.q.cpu().numpy(), q) and np.array_equal(ck.scale.cpu().numpy(), s)


def norm_dx_tol(dy, x, st, gain):
    """g and xh are off by 3 u each, the two means by depth u; each of the three terms by 3 u more."""
    rstd = st[:, 1:]
    xh, g = np.abs(x - st[:, :1]) * rstd, np.abs(dy) * (1.0 if gain is None else np.abs(gain))
    return rstd * (DEPTH + 12) * U * (g + g.mean(1, keepdims=True) + xh * (g * xh).mean(1, keepdims=True))


@pytest.mark.parametrize("rows,cols", NORM_SHAPES)
@pytest.mark.parametrize("kind,dyd,affine,off", [("f32", F32, True, 0), ("bf16", BF16, True, 1), ("ckpt", BF16, True, 0), ("ckpt", F32, False, 1),
                                                 ("bf16", F32, True, 0), ("f32", BF16, False, 3)])
def test_layernorm_backward(rows, cols, kind, dyd, affine, off):
    say("layernorm_backward", rows, cols, kind, dyd, affine, off)
    x, gain, _ = norm_inputs(rows, cols, F32 if kind == "f32" else BF16, 30)
    gain = gain if affine else None
    _, stats = ma.layernorm_forward(x)
    dy = rand((rows, cols), 34, dyd, 0.1)
    xin, xn = x, f64(x)
    if kind == "ckpt":
        xin = ma.act_pack(x)
        xn = T.act_unpack(*T.act_pack(xn), cols)
    else:
        _, xin = view(x, off)
    st = f64(stats)
    dx, dgain, dbias = T.layernorm_backward(f64(dy), xn, st[:, :1], st[:, 1:], None if gain is None else f64(gain))
    _, dyv = view(dy, off)
    dxd = dyd if kind == "ckpt" else x.dtype
    db, dxv = view(torch.zeros(rows, cols, dtype=dxd, device=DEV), off)
    g0, b0 = rand((cols,), 35), rand((cols,), 36)
    gg, gb = g0.clone(), b0.clone()
    ma.layernorm_backward(dyv, xin, stats, gain, dgain=gg, dbias=gb, dx=dxv)
    xh = np.abs(xn - st[:, :1]) * st[:, 1:]
    close(dxv, dx, norm_dx_tol(f64(dy), xn, st, f64(gain) if affine else None), dxd)
    assert guards(db, rows * cols, off)
    # a column's sum: every row one addition at most, products off by 4 u
    n = rows + 40
    mg, mb = (np.abs(f64(dy)) * xh).sum(0), np.abs(f64(dy)).sum(0)
    close(gg, dgain, (n + 4) * U * mg)
    close(gb, dbias, n * U * mb)
    ag, ab = g0.clone(), b0.clone()
    dx2 = ma.layernorm_backward(dy, xin, stats, gain, dgain=ag, dbias=ab, accumulate=True)
    assert torch.equal(dx2, dxv) and torch.equal(ag, g0 + gg) and torch.equal(ab, b0 + gb)
    only = torch.empty_like(b0)
    assert torch.equal(ma.layernorm_backward(dy, xin, stats, gain, dbias=only), dxv) and torch.equal(only, gb)
    assert torch.equal(ma.layernorm_backward(dy, xin, stats, gain), dxv)


def test_layernorm_many_rows_sum_every_row_once():
    rows, cols = 5003, 96
    x, dy = rand((rows, cols), 40, BF16), torch.ones(rows, cols, dtype=BF16, device=DEV)
    _, stats = ma.layernorm_forward(x)
    dg, db = torch.empty(cols, device=DEV), torch.empty(cols, device=DEV)
    ma.layernorm_backward(dy, x, stats, dgain=dg, dbias=db)
    assert bool((db == rows).all())
    xh = (f64(x) - f64(stats)[:, :1]) * f64(stats)[:, 1:]
    close(dg, xh.sum(0), (rows + 44) * U * np.abs(xh).sum(0))


def test_layernorm_without_rows():
    x = torch.empty(0, 64, device=DEV)
    y, stats = ma.layernorm_forward(x)
    assert y.shape == (0, 64) and stats.shape == (0, 2)
    dg = torch.ones(64, device=DEV)
    assert ma.layernorm_backward(y, x, stats, dgain=dg, accumulate=True).shape == (0, 64) and bool((dg == 1).all())
    ma.layernorm_backward(y, x, stats, dgain=dg)
    assert not dg.any()


@pytest.mark.parametrize("eps", [1e-40, 1e-30])
def test_layernorm_of_equal_values_with_a_tiny_eps(eps):
    """A row of equal values has no variance: y is the bias and rstd 1 / sqrt(eps), also where eps is subnormal."""
    x, b = torch.full((5, 256), 0.5, device=DEV), rand((256,), 44)
    y, stats = ma.layernorm_forward(x, bias=b, eps=eps)
    assert torch.equal(y, b.expand(5, 256))
    want = 1.0 / np.sqrt(float(np.float32(eps)))
    # the reciprocal root is good to 2 units in the last place
    close(stats[:, 1], np.full(5, want), 4 * U * want)


def test_layernorm_nonfinite_rows_stay_in_their_row():
    x = rand((6, 700), 41)
    x[2, 13], x[4, 699] = float("nan"), float("inf")
    y, stats = ma.layernorm_forward(x)
    bad = torch.isnan(y).all(1).cpu()
    assert bad.tolist() == [False, False, True, False, True, False]
    ok = [0, 1, 3, 5]
    y2, s2 = ma.layernorm_forward(x[ok].contiguous())
    assert torch.equal(y[ok], y2) and torch.equal(stats[ok], s2)


def test_layernorm_gradient_against_differences():
    """dx, dgain and dbias against central differences of the fp64 formula along random directions."""
    rows, cols = 4, 200
    x, gain, bias = norm_inputs(rows, cols, F32, 50)
    x[1] = rand((cols,), 54)
    dy = rand((rows, cols), 55)
    _, stats = ma.layernorm_forward(x, gain, bias)
    dg, db = torch.empty(cols, device=DEV), torch.empty(cols, device=DEV)
    dx = ma.layernorm_backward(dy, x, stats, gain, dgain=dg, dbias=db)
    f = lambda x, g, b: (T.layernorm_forward(x, g, b)[0] * f64(dy)).sum()  # noqa: E731
    rng, h = np.random.default_rng(0), 1e-5
    base = [f64(x), f64(gain), f64(bias)]
    for k, grad in enumerate((dx, dg, db)):
        v = rng.standard_normal(base[k].shape)
        p, m = list(base), list(base)
        p[k], m[k] = base[k] + h * v, base[k] - h * v
        diff = (f(*p) - f(*m)) / (2 * h)
        # the kernel's gradient is off by its bound times |v|; the quotient by the third derivative's h^2 / 6, with
        # row deviations near 1 some 1e-10 of |y dy|, and by the rounding of f, 2^-52 of sum |y dy| over h
        own = [norm_dx_tol(f64(dy), f64(x), f64(stats), f64(gain)), (rows + 44) * U * np.abs(f64(dy) * 6.0).sum(0),
               (rows + 40) * U * np.abs(f64(dy)).sum(0)][k]   # |xh| < 6 here
        mag = np.abs(T.layernorm_forward(*base)[0] * f64(dy)).sum()
        assert abs(diff - (f64(grad) * v).sum()) <= (own * np.abs(v)).sum() + (2.0 ** -52 / h * 16 + 1e-8) * mag


# ---------------------------------------------------------------------------
# checkpoints
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 7), (2, 128), (5, 129), (17, 1000), (64, 1024), (3, 4099), (257, 136)])
@pytest.mark.parametrize("dt,off", [(F32, 0), (BF16, 0), (BF16, 1), (F32, 3)])
def test_checkpoint_bits(rows, cols, dt, off):
    say("checkpoint", rows, cols, dt, off)
    rng = np.random.default_rng(rows * cols)
    x = rng.standard_normal((rows, cols)) * 2.0 ** rng.integers(-140, 126, (rows, 1))
    x[rng.random((rows, cols)) < 0.1] = 0.0
    x.flat[:: 97] *= -2.0 ** -20
    x = torch.from_numpy(x).float().to(dt).to(DEV)
    if rows > 2:
        x[1] = 0
        x[2, 0], x[2, -1], x[2, cols // 2] = float("inf"), float("-inf"), float("nan")
        x[0, 0] = torch.finfo(dt).max
    xb, xv = view(x, off)
    c = ma.act_pack(xv)
    q, s = T.act_pack(f64(x))
    got = c.q.cpu().numpy()
    nan = (q & 127) == 127
    assert np.array_equal(np.where(nan, got & 127, got), np.where(nan, 127, q)) and np.array_equal(c.scale.cpu().numpy(), s)
    for od in (F32, BF16):
        ob, ov = view(torch.zeros(rows, cols, dtype=od, device=DEV), off)
        ma.act_unpack(c, out=ov)
        assert np.array_equal(to_np(ov), T.act_unpack(q, s, cols).astype(np.float32), equal_nan=True) and guards(ob, rows * cols, off)
    assert guards(xb, rows * cols, off)


def test_checkpoint_rounds_every_bf16_value_as_defined():
    """All 65536 bf16 patterns, each beside every magnitude class of block maximum."""
    v = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(BF16)
    for k in range(0, 256, 5):
        x = v.view(512, 128).clone()
        top = torch.tensor([k << 7], dtype=torch.int32).to(torch.int16).view(BF16)
        x[:, 0] = top if k < 255 else 0
        c = ma.act_pack(x.to(DEV))
        q, s = T.act_pack(f64(x))
        got, nan = c.q.cpu().numpy(), (q & 127) == 127
        assert np.array_equal(np.where(nan, got & 127, got), np.where(nan, 127, q)) and np.array_equal(c.scale.cpu().numpy(), s)


def test_checkpoint_of_leading_dimensions_and_reuse():
    x = rand((2, 3, 200), 60, BF16)
    c = ma.act_pack(x)
    assert (c.rows, c.cols, c.nbytes()) == (6, 200, 6 * 256 + 6 * 2)
    assert torch.equal(ma.act_unpack(c, out=torch.empty(2, 3, 200, device=DEV)).view(6, 200), ma.act_unpack(c, dtype=F32))
    before = ma.act_unpack(c)
    assert ma.act_pack(x * 2, out=c) is c and torch.equal(ma.act_unpack(c), before * 2)
    e = ma.act_pack(x[:0])
    assert e.rows == 0 and ma.act_unpack(e).shape == (0, 200)


# ---------------------------------------------------------------------------
# weight gradient
# ---------------------------------------------------------------------------
WGRAD = [(1, 1, 1), (2, 8, 128), (7, 5, 3), (63, 64, 128), (64, 65, 129), (65, 255, 257), (1000, 250, 333), (128, 256, 256),
         (129, 264, 384), (300, 520, 640), (4096, 64, 128), (2500, 136, 200), (5000, 7, 512), (33, 1000, 17)]


@pytest.mark.parametrize("t,n,k", WGRAD)
@pytest.mark.parametrize("dyd,gd,acc,off", [(BF16, BF16, False, 0), (BF16, F32, True, 0), (F32, F32, False, 0), (F32, BF16, True, 1), (BF16, BF16, True, 1)])
def test_weight_grad(t, n, k, dyd, gd, acc, off):
    say("weight_grad", t, n, k, dyd, gd, acc, off)
    dy, x = rand((t, n), 70, dyd, 0.1), rand((t, k), 71, BF16)
    x *= 2.0 ** torch.randint(-6, 6, (t, 1), device=DEV)
    c = ma.act_pack(x)
    g0 = rand((n, k), 72, gd)
    want, mag = T.act_weight_grad(f64(dy), f64(ma.act_unpack(c)), f64(g0) if acc else None)
    _, dyv = view(dy, off)
    gb, gv = view(g0, off)
    ma.act_weight_grad(dyv, c, gv, accumulate=acc)
    # fp32 dy enters as three bf16 terms: 3 t additions; 2 u each leaves room for a unit that truncates
    tol = ((3 if dyd == F32 else 1) * t + 16) * 2 * U * mag + (U * (np.abs(f64(g0)) + mag) if acc else 0)
    close(gv, want, tol, gd)
    assert guards(gb, n * k, off)
    again = g0.clone()
    ma.act_weight_grad(dy, c, again, accumulate=acc)
    assert torch.equal(again, gv)


def test_weight_grad_is_exact_for_exact_sums():
    """Small whole numbers: every sum is exact, so an element in a wrong place or counted twice shows."""
    for t, n, k in ((200, 300, 290), (777, 129, 513), (1024, 512, 512)):
        g = torch.Generator().manual_seed(t)
        dy = torch.randint(-4, 5, (t, n), generator=g).float()
        x = torch.randint(-8, 9, (t, k), generator=g).float()
        want = (dy.double().t() @ x.double()).float()
        c = ma.act_pack(x.to(DEV))
        assert torch.equal(ma.act_unpack(c, dtype=F32).cpu(), x)
        for dyd in (F32, BF16):
            got = ma.act_weight_grad(dy.to(dyd).to(DEV), c, torch.empty(n, k, device=DEV))
            assert torch.equal(got.cpu(), want)


def test_weight_grad_keeps_fp32_precision_of_dy():
    """dy with 24 significant bits against one-hot activations: the gradient is dy itself."""
    t = 96
    dy = rand((t, 70), 73)
    c = ma.act_pack(torch.eye(t, device=DEV))
    got = ma.act_weight_grad(dy, c, torch.empty(70, t, device=DEV))
    assert torch.equal(got, dy.t().contiguous())


def test_weight_grad_of_no_tokens_and_nonfinite_values():
    c = ma.ActCheckpoint.empty(0, 200, DEV)
    g = torch.ones(30, 200, device=DEV)
    ma.act_weight_grad(torch.empty(0, 30, device=DEV), c, g, accumulate=True)
    assert bool((g == 1).all())
    ma.act_weight_grad(torch.empty(0, 30, device=DEV), c, g)
    assert not g.any()
    # a NaN or infinity in dy reaches its own row of the gradient only, one in x its own column only
    for dt in (BF16, F32):
        for t in (70, 64):
            dy, x = rand((t, 300), 74, dt), rand((t, 300), 75, BF16).abs() + 0.1
            clean = ma.act_weight_grad(dy, ma.act_pack(x), torch.empty(300, 300, device=DEV))
            dy[t - 1, 299], dy[0, 7], x[3, 130] = float("inf"), float("nan"), float("nan")
            got = ma.act_weight_grad(dy, ma.act_pack(x), torch.empty(300, 300, device=DEV))
            fin = torch.isfinite(got)
            want = torch.ones(300, 300, dtype=torch.bool, device=DEV)
            want[299], want[7], want[:, 130] = False, False, False
            assert torch.equal(fin, want)
            # dropping NaN from a block changes no scale here unless it was its maximum
            assert torch.equal(got[:, :128][want[:, :128]], clean[:, :128][want[:, :128]])


# ---------------------------------------------------------------------------
# streams, graphs, and the run of them together
# ---------------------------------------------------------------------------
def _every(n, seed=80):
    """One call of every operator on n tokens: (run, inputs)."""
    w, t = rand((500, 264), seed), tokens("zipf", 500, n, seed + 1).to(DEV)
    gain, bias = 1 + rand((264,), seed + 2, F32, 0.1), rand((264,), seed + 3, F32, 0.1)
    dw = rand((136, 264), seed + 4)
    ge, gg, gb = torch.empty(500, 264, device=DEV), torch.empty(264, device=DEV), torch.empty(264, device=DEV)
    dy = rand((n, 136), seed + 5, BF16)

    def run(stream=None):
        x = ma.embedding_forward(w, t, scale=3.0, dtype=BF16, stream=stream)
        ck = ma.ActCheckpoint.empty(n, 264, DEV)
        y, stats = ma.layernorm_forward(x, gain, bias, checkpoint=ck, stream=stream)
        yc = ma.act_pack(y, stream=stream)
        ma.act_weight_grad(dy, yc, dw, stream=stream)
        dx = ma.layernorm_backward(y, ck, stats, gain, dgain=gg, dbias=gb, stream=stream)
        ma.embedding_backward(dx, t, ge, scale=3.0, stream=stream)
        return [dw, gg, gb, ge, dx, ma.act_unpack(yc, stream=stream)]
    return run, (w, t, dy)


# in one launch, and through the sort and the joins
BOTH = pytest.mark.parametrize("n", [700, 1500])


@BOTH
def test_another_stream_gives_the_same_bits(n):
    run, _ = _every(n)
    want = [x.clone() for x in run()]
    torch.cuda.synchronize()
    s = torch.cuda.Stream(DEV)
    for how in (s, s.cuda_stream):
        got = run(how)
        s.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    with torch.cuda.stream(s):
        got = run()
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@BOTH
def test_graph_replays_match_eager_calls(n):
    run, (w, t, dy) = _every(n)
    run2, (w2, t2, dy2) = _every(n)
    side = torch.cuda.Stream(DEV)
    with torch.cuda.stream(side):
        run2()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run2()
    for i in range(4):
        new = tokens("zipf", 500, n, 90 + i).to(DEV)
        t.copy_(new)
        t2.copy_(new)
        w2.mul_(1.25)
        w.mul_(1.25)
        want = run()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want)), i


@BOTH
def test_two_streams_at_once(n):
    (a, _), (b, _) = _every(n, 80), _every(n, 180)
    wa, wb = [x.clone() for x in a()], [x.clone() for x in b()]
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(DEV), torch.cuda.Stream(DEV)
    for _ in range(3):
        with torch.cuda.stream(s1):
            ga = a()
        with torch.cuda.stream(s2):
            gb = b()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(ga, wa)) and all(torch.equal(x, y) for x, y in zip(gb, wb))


def test_offsets_past_32_bits():
    """Operands of more than 2^32 bytes: the last rows give what a call on them alone gives."""
    n, cols, last = (1 << 21) + 1000, 2048, 700
    x = torch.empty(n, cols, dtype=BF16, device=DEV)
    x.view(torch.int16).fill_(0x3F81)                    # not quite 1
    x[-last:] = rand((last, cols), 110, BF16)
    ck, gain = ma.ActCheckpoint.empty(n, cols, DEV), 1 + rand((cols,), 111, F32, 0.1)
    y, stats = ma.layernorm_forward(x, gain, checkpoint=ck)
    small = ma.ActCheckpoint.empty(last, cols, DEV)
    ys, ss = ma.layernorm_forward(x[-last:], gain, checkpoint=small)
    assert torch.equal(y[-last:], ys) and torch.equal(stats[-last:], ss)
    assert torch.equal(ck.q[-last:], small.q) and torch.equal(ck.scale[-last:], small.scale)
    packed = ma.act_pack(x)
    assert torch.equal(packed.q[-last:], small.q) and torch.equal(packed.scale, ck.scale)
    assert torch.equal(ma.act_unpack(packed, out=y)[-last:], ma.act_unpack(small))
    for held, alone in ((x, x[-last:]), (ck, small)):
        dx = ma.layernorm_backward(x, held, stats, gain, dx=y)
        assert torch.equal(dx[-last:], ma.layernorm_backward(x[-last:], alone, ss, gain))
    # a weight gradient whose only nonzero dy are in the last rows
    x[:-last] = 0
    dw = ma.act_weight_grad(x, ma.ActCheckpoint(packed.q[:, :128].contiguous(), packed.scale[:, :1].contiguous(), 128),
                            torch.empty(cols, 128, device=DEV))
    want, mag = T.act_weight_grad(f64(x[-last:]), f64(ma.act_unpack(small)[:, :128]))
    close(dw, want, 2 * (last + 16) * U * mag)
    # a table's last rows, looked up by the last tokens
    t = torch.full((n,), -1, device=DEV)
    t[-last:] = n - 1 - torch.arange(last, device=DEV) // 2
    assert torch.equal(ma.embedding_forward(x, t, out=y)[-last:], x[t[-last:]]) and not y[:-last].any()
    del y, ck, packed
    grad = ma.embedding_backward(x, t, torch.empty(n, cols, device=DEV))
    pairs = x[-last:].float().view(-1, 2, cols)
    assert torch.equal(grad[-last // 2:].flip(0), pairs[:, 0] + pairs[:, 1]) and not grad[:-last // 2].any()


@pytest.mark.parametrize("cols", [1023, 1025, 1026])
def test_large_calls_with_ragged_rows(cols):
    """Calls that pass the caches (more than 192 MB) give what calls on some of their rows give."""
    n, pick = 60000, torch.tensor([0, 1, 777, 31000, 59998, 59999], device=DEV)
    for dt in (F32, BF16):
        buf, x = view(rand((n, cols), 120, dt), 1)
        for od in (F32, BF16):
            ob, y = view(torch.zeros(n, cols, dtype=od, device=DEV), 1)
            ck, few = ma.ActCheckpoint.empty(n, cols, DEV), ma.ActCheckpoint.empty(6, cols, DEV)
            _, stats = ma.layernorm_forward(x, out=y, checkpoint=ck)
            ys, ss = ma.layernorm_forward(x[pick].contiguous(), dtype=od, checkpoint=few)
            # other lanes per row, so other orders of the sums: either value is off by DEPTH u (E|x| + 2 |y|), with
            # E|x| < 1 and |y| < 6, and rounded once
            close(y[pick], f64(ys), 26 * DEPTH * U + half(od) * np.abs(f64(ys)), od)
            assert torch.equal(ck.q[pick], few.q) and torch.equal(ck.scale[pick], few.scale)
            assert guards(ob, n * cols, 1)
            assert torch.equal(ma.act_pack(x).q, ck.q)
            assert torch.equal(ma.act_unpack(ck, out=y)[pick], ma.act_unpack(few, dtype=od)) and guards(ob, n * cols, 1)
            t = torch.randint(0, n, (n,), device=DEV, generator=torch.Generator(DEV).manual_seed(121))
            assert torch.equal(ma.embedding_forward(x, t, out=y), x[t].to(od)) and guards(ob, n * cols, 1)
        gb, g = view(torch.ones(n, cols, device=DEV), 1)
        p = torch.randperm(n, device=DEV, generator=torch.Generator(DEV).manual_seed(122))[:5000]
        ma.embedding_backward(x[:5000], p, g)
        assert torch.equal(g[p], x[:5000].float()) and guards(gb, n * cols, 1)
        g[p] = 0
        assert not g.any()


def test_training_step_end_to_end():
    """Embedding, norm with checkpoint, a linear layer, their gradients out of the checkpoints, and the optimizer
    step that reads them, against the same chain in fp64 from the stored values of each stage."""
    rows, cols, outs, n = 300, 256, 512, 640
    table, W = rand((rows, cols), 100, F32, 0.5), rand((outs, cols), 101, BF16, 0.05)
    gain, bias = torch.ones(cols, device=DEV), torch.zeros(cols, device=DEV)
    t = tokens("zipf", rows, n, 102).to(DEV)
    x = ma.embedding_forward(table, t, scale=16.0, dtype=BF16)
    ck = ma.ActCheckpoint.empty(n, cols, DEV)
    y, stats = ma.layernorm_forward(x, gain, bias, checkpoint=ck)
    yc = ma.act_pack(y)
    z = y.float() @ W.float().t()
    dz = (z / n).bfloat16()                              # loss = |z|^2 / 2n
    gW = torch.empty(1, outs, cols, dtype=BF16, device=DEV)
    ma.act_weight_grad(dz, yc, gW[0])
    dyv = (dz.float() @ W.float()).bfloat16()
    gg, gb, gt = torch.empty(cols, device=DEV), torch.empty(cols, device=DEV), torch.empty(rows, cols, device=DEV)
    dx = ma.layernorm_backward(dyv, ck, stats, gain, dgain=gg, dbias=gb)
    ma.embedding_backward(dx, t, gt, scale=16.0)
    # each gradient against fp64 on the same stored inputs
    want, mag = T.act_weight_grad(f64(dz), f64(ma.act_unpack(yc)))
    close(gW[0], want, 2 * (n + 16) * U * mag, BF16)
    xs, st = f64(ma.act_unpack(ck)), f64(stats)
    rdx, rdg, rdb = T.layernorm_backward(f64(dyv), xs, st[:, :1], st[:, 1:], f64(gain))
    close(dx, rdx, norm_dx_tol(f64(dyv), xs, st, f64(gain)), BF16)
    wt, mt, count = T.embedding_backward(f64(dx), t.cpu().numpy(), rows, 16.0)
    close(gt, wt, (count[:, None] * 1.02 + 3) * U * mt)
    # and the step itself: finite, and it moves what has a gradient
    W1, table1 = W.clone().view(1, outs, cols), table.clone()
    M = torch.zeros(1, outs, cols, dtype=BF16, device=DEV)
    seg = [dict(param=p, grad=g, exp_avg=torch.zeros_like(p), exp_avg_sq=torch.zeros_like(p), lr=1e-3, step=1)
           for p, g in ((table1.view(-1), gt.view(-1)), (gain.clone(), gg), (bias.clone(), gb))]
    ma.optimizer_step([ma.MuonGroup(W1, gW, M)], ma.MuonHParams(lr=0.02), seg)
    torch.cuda.synchronize()
    touched = torch.from_numpy(count > 0).to(DEV)
    assert torch.isfinite(W1.float()).all() and not torch.equal(W1[0], W)
    assert torch.equal(table1[~touched], table[~touched]) and bool((table1[touched] != table[touched]).any(1).all())


# ---------------------------------------------------------------------------
# rows of equal values: the mean is the value itself, whatever 1 / cols rounds to
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("rows", [5, 600])
@pytest.mark.parametrize("cols", [1, 3, 41, 82, 333, 1000, 1025, 2047, 4099, 8200, 16383])
@pytest.mark.parametrize("xd,yd", [(F32, F32), (BF16, F32), (F32, BF16), (BF16, BF16)])
def test_layernorm_of_equal_values(rows, cols, xd, yd):
    """x - mean is a small multiple of x's step in every column, so its sum and the sum over cols are exact: the
    corrected mean is x, the variance 0, y the bias and rstd that of eps alone."""
    say("layernorm of equal values", rows, cols, xd, yd)
    values = torch.tensor([0.5, 1000.1, -3.3e7, 1e-3, 1e15], device=DEV).to(xd)
    x = values[torch.arange(rows, device=DEV) % 5, None].expand(rows, cols).contiguous()
    bias, gain = rand((cols,), 130), 1 + rand((cols,), 131)
    for eps in (1e-5, 1e-30):
        y, stats = ma.layernorm_forward(x, gain, bias, eps=eps, dtype=yd)
        assert torch.equal(stats[:, 0], x[:, 0].float())
        assert torch.equal(y, bias.to(yd).expand(rows, cols))
        want = 1.0 / np.sqrt(float(np.float32(eps)))
        close(stats[:, 1], np.full(rows, want), 4 * U * want)   # (the reciprocal root: 2 units in the last place)


def test_layernorm_mean_of_a_row_with_an_infinity():
    """The mean of a row with an infinity is that infinity, also behind the correction of the mean."""
    x = rand((4, 700), 132)
    x[1, 5], x[3, 699] = float("inf"), float("-inf")
    _, stats = ma.layernorm_forward(x)
    assert stats[1, 0].item() == float("inf") and stats[3, 0].item() == float("-inf")
    assert torch.isnan(stats[[1, 3], 1]).all() and torch.isfinite(stats[[0, 2]]).all()


# ---------------------------------------------------------------------------
# both tiles of the weight gradient, each with one split of the tokens and with several: (tokens, outs, ins, edge of
# the tile, splits or None for several, dy's types that take it there)
# ---------------------------------------------------------------------------
TILES = [
    (5, 4090, 4081, 256, 1, (BF16, F32)), (65, 1030, 8200, 256, 1, (BF16, F32)), (130, 4096, 4096, 256, 1, (BF16, F32)),
    (700, 4090, 4081, 256, 1, (BF16, F32)), (4099, 2050, 2041, 256, None, (BF16, F32)), (8192, 3000, 1000, 256, None, (BF16, F32)),
    (1000, 2041, 2050, 256, None, (F32,)), (1000, 2050, 2041, 128, 1, (BF16,)), (63, 130, 300, 128, 1, (BF16,)),
    (4096, 64, 128, 128, None, (BF16, F32)), (1000, 250, 333, 128, None, (BF16, F32)), (20, 250, 333, 128, 1, (BF16, F32)),
]
EVERY_TILE = [(*case[:5], dt) for case in TILES for dt in case[5]]


def assert_tile(t, n, k, edge, splits, dyd):
    e, s = C.c_int32(), C.c_int32()
    L.check(L.lib().ma_test_act_weight_grad_plan(t, n, k, L.MA_F32 if dyd == F32 else L.MA_BF16, C.byref(e), C.byref(s)))
    assert e.value == edge and (s.value > 1 if splits is None else s.value == splits), (e.value, s.value)


def product(dy, x):
    """dy^T x in fp64 on the device."""
    return dy.double().t().contiguous() @ x.double()


def close_on_device(got, want, tol, dtype):
    """As `close`, of finite fp64 tensors."""
    bound = tol * (1 + half(dtype)) + half(dtype) * want.abs() + torch.finfo(dtype).smallest_normal * half(dtype) * 2
    assert bool(((got.double() - want).abs() <= bound).all())


@pytest.mark.parametrize("t,n,k,edge,splits,dyd", EVERY_TILE)
@pytest.mark.parametrize("gd,acc,off", [(F32, False, 1), (BF16, True, 0), (F32, True, 0), (BF16, False, 3)])
def test_weight_grad_of_every_tile(t, n, k, edge, splits, dyd, gd, acc, off):
    say("weight_grad tile", t, n, k, edge, splits, dyd, gd, acc, off)
    assert_tile(t, n, k, edge, splits, dyd)
    dy, x = rand((t, n), 140, dyd, 0.1), rand((t, k), 141, BF16)
    x *= 2.0 ** torch.randint(-6, 6, (t, 1), device=DEV)
    c = ma.act_pack(x)
    held, g0 = ma.act_unpack(c), rand((n, k), 142, gd)
    want, mag = product(dy, held), product(dy.abs(), held.abs())
    _, dyv = view(dy, off)
    gb, gv = view(g0, off)
    ma.act_weight_grad(dyv, c, gv, accumulate=acc)
    # as in test_weight_grad: t additions, three times as many for fp32 dy, 2 u each
    tol = ((3 if dyd == F32 else 1) * t + 16) * 2 * U * mag
    if acc:
        want, tol = want + g0.double(), tol + U * (g0.double().abs() + mag)
    close_on_device(gv, want, tol, gd)
    assert guards(gb, n * k, off)
    again = g0.clone()
    ma.act_weight_grad(dy, c, again, accumulate=acc)
    assert torch.equal(again, gv)


@pytest.mark.parametrize("t,n,k,edge,splits,dyd", EVERY_TILE)
def test_weight_grad_of_every_tile_is_exact_for_exact_sums(t, n, k, edge, splits, dyd):
    """Small whole numbers: every sum is exact, so an element in a wrong place or counted twice shows."""
    say("weight_grad tile, whole numbers", t, n, k, edge, splits, dyd)
    assert_tile(t, n, k, edge, splits, dyd)
    g = torch.Generator(DEV).manual_seed(t + n)
    dy = torch.randint(-4, 5, (t, n), generator=g, device=DEV).to(dyd)
    x = torch.randint(-8, 9, (t, k), generator=g, device=DEV).float()
    got = ma.act_weight_grad(dy, ma.act_pack(x), torch.empty(n, k, device=DEV))
    assert torch.equal(got.double(), product(dy, x))


@pytest.mark.parametrize("t,n,k,edge,splits,dyd", [c for c in EVERY_TILE if c[0] >= 20 and c[2] >= 300])
def test_weight_grad_of_every_tile_keeps_nonfinite_values_in_their_places(t, n, k, edge, splits, dyd):
    """A NaN or infinity in dy reaches its own row of the gradient only, one in x its own column only."""
    say("weight_grad tile, nonfinite", t, n, k, edge, splits, dyd)
    assert_tile(t, n, k, edge, splits, dyd)
    dy, x = rand((t, n), 143, dyd), rand((t, k), 144, BF16).abs() + 0.1
    dy[t - 1, n - 1], dy[0, 7], x[3, k - 1] = float("inf"), float("nan"), float("nan")
    got = ma.act_weight_grad(dy, ma.act_pack(x), torch.empty(n, k, device=DEV))
    want = torch.ones(n, k, dtype=torch.bool, device=DEV)
    want[n - 1], want[7], want[:, k - 1] = False, False, False
    assert torch.equal(torch.isfinite(got), want)


def test_both_tiles_ran_with_one_split_and_with_several():
    ran = {(edge, splits == 1, dyd) for _, _, _, edge, splits, dyd in EVERY_TILE}
    assert len(ran) == 8


# ---------------------------------------------------------------------------
# more than 1024 rows of more than 8192 columns: operands read twice, and partial sums
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("rows,cols", [(1030, 8200), (1100, 16383), (1025, 16384)])
@pytest.mark.parametrize("kind,dyd,affine,off", [("f32", F32, True, 0), ("bf16", BF16, True, 1), ("ckpt", F32, False, 1), ("ckpt", BF16, True, 0)])
def test_layernorm_backward_of_many_wide_rows(rows, cols, kind, dyd, affine, off):
    assert ma.layernorm_workspace_size(rows, cols) > 0
    test_layernorm_backward(rows, cols, kind, dyd, affine, off)


# ---------------------------------------------------------------------------
# token ids that only their upper 32 bits, or the sign of the lower ones, keep out of the table
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("rows,cols,n", [(50, 24, 5), (300, 40, 64), (300, 40, 700), (97, 530, 1024), (97, 530, 1025),
                                         (1000, 72, 5003), (300, 16, 16384), (700, 8, 40000)])
@pytest.mark.parametrize("acc", [False, True])
def test_embedding_gradient_of_far_tokens(rows, cols, n, acc):
    say("embedding gradient of far tokens", rows, cols, n, acc)
    g = torch.Generator().manual_seed(150)
    r, d = torch.randint(0, rows, (n,), generator=g), rand((n, cols), 151)
    far = torch.tensor([0, 1 << 32, 1 << 40, -(1 << 32), -(1 << 40), (1 << 31) - rows, 1 << 31, 3 << 30, -(1 << 63)])
    which = torch.randint(0, 9, (n,), generator=g)
    which[::3] = 0
    t = r + far[which]
    d[(t != r).to(DEV)] = float("nan")              # what is ignored is not read
    g0 = rand((rows, cols), 152)
    got = ma.embedding_backward(d, t.to(DEV), g0.clone(), accumulate=acc)
    want, mag, count = T.embedding_backward(np.nan_to_num(f64(d)), t.numpy(), rows, 1.0, f64(g0) if acc else None)
    assert 0 < count.sum() < n
    # as in test_embedding_backward
    close(got, want, (count[:, None] * (1 + 1 / 64) + 3) * U * mag + (U * (np.abs(f64(g0)) + mag) if acc else 0))


@pytest.mark.parametrize("rows,cols", [(1000, 40), (50304, 24)])
def test_embedding_workspace_serves_fewer_tokens_too(rows, cols):
    """One workspace, of the size for the longest batch, for every shorter one."""
    longest = 20000
    ws = torch.empty(ma.embedding_workspace_size(rows, cols, longest), dtype=torch.uint8, device=DEV)
    t, d = tokens("zipf", rows, longest, 160).to(DEV), rand((longest, cols), 161, BF16)
    for n in (longest, 16385, 16384, 3000, 1025, 1024, 5):
        say("embedding workspace", rows, cols, n)
        got = ma.embedding_backward(d[:n], t[:n], torch.empty(rows, cols, device=DEV), workspace=ws)
        assert torch.equal(got, ma.embedding_backward(d[:n], t[:n], torch.empty(rows, cols, device=DEV)))


def test_weight_grad_of_small_fp32_dy():
    """dy against one-hot activations is all there from 2^-110 up; below, what three terms of bf16 leave is under
    2^-133, bf16's least number, whose multiples add up exactly in fp32."""
    t, g = 96, torch.Generator().manual_seed(170)
    m = (1 + torch.rand(t, 70, generator=g, dtype=torch.float64)) * torch.where(torch.rand(t, 70, generator=g) < 0.5, -1.0, 1.0)
    for s in (0, 60):
        c = ma.act_pack(torch.eye(t, device=DEV) * 2.0 ** s)
        for e in (-90, -105, -110, -112, -118, -124, -126, -128, -132):
            dy = (m * 2.0 ** e).float()
            got = ma.act_weight_grad(dy.to(DEV), c, torch.empty(70, t, device=DEV)).cpu().double() * 2.0 ** -s
            off = (got - dy.t().double()).abs()
            assert not off.any() if e >= -110 else bool((off < 2.0 ** -133).all()), (s, e)


def test_operators_stand_outside_autograd():
    """Inputs that require grad are read as data: the same bits, no graph, no gradient. In a Function of the caller's
    the backward calls give the gradients that autograd then passes on."""
    w, t, gain = rand((40, 96), 180), tokens("spread", 40, 50, 181).to(DEV), 1 + rand((96,), 182, F32, 0.1)
    plain = ma.embedding_forward(w, t)
    want, stats = ma.layernorm_forward(plain, gain)
    wg, gg = w.clone().requires_grad_(), gain.clone().requires_grad_()
    x = ma.embedding_forward(wg, t)
    y, _ = ma.layernorm_forward(x, gg)
    assert torch.equal(x, plain) and torch.equal(y, want) and not x.requires_grad and not y.requires_grad

    class Norm(torch.autograd.Function):
        @staticmethod
        def forward(ctx, w, gain):
            x = ma.embedding_forward(w, t)
            y, stats = ma.layernorm_forward(x, gain)
            ctx.save_for_backward(x, stats, gain)
            return y

        @staticmethod
        def backward(ctx, dy):
            x, stats, gain = ctx.saved_tensors
            dgain = torch.empty_like(gain)
            dx = ma.layernorm_backward(dy.contiguous(), x, stats, gain, dgain=dgain)
            return ma.embedding_backward(dx, t, torch.empty_like(w)), dgain

    dy = rand((50, 96), 183)
    Norm.apply(wg, gg).backward(dy)
    dgain = torch.empty_like(gain)
    dx = ma.layernorm_backward(dy, plain, stats, gain, dgain=dgain)
    assert torch.equal(gg.grad, dgain) and torch.equal(wg.grad, ma.embedding_backward(dx, t, torch.empty_like(w)))


# ---------------------------------------------------------------------------
# the largest rows and columns that each operator takes, with few of the other
# ---------------------------------------------------------------------------
def whole(shape, seed, dtype, most=4):
    """Small whole numbers, whose sums are exact."""
    return torch.randint(-most, most + 1, shape, generator=torch.Generator(DEV).manual_seed(seed), device=DEV).to(dtype)


@pytest.mark.parametrize("n", [900, 1500])
def test_largest_table(n):
    rows = 1 << 24
    say("largest table", n)
    w = rand((rows, 2), 190)
    t = 1 + torch.randperm(rows - 2, generator=torch.Generator(DEV).manual_seed(191), device=DEV)[:n]
    t[0], t[1] = rows - 1, 0
    assert torch.equal(ma.embedding_forward(w, t), w[t])
    d = rand((n, 2), 192)
    g = ma.embedding_backward(d, t, torch.empty_like(w))
    assert torch.equal(g[t], d)
    g[t] = 0
    assert not g.any()


@pytest.mark.parametrize("n", [20, 1030])
def test_widest_table(n):
    cols = 1 << 20
    say("widest table", n)
    w, t = whole((3, cols), 193, BF16), torch.randint(0, 3, (n,), generator=torch.Generator(DEV).manual_seed(194), device=DEV)
    assert torch.equal(ma.embedding_forward(w, t[:20], dtype=F32), w[t[:20]].float())
    d = whole((n, cols), 195, BF16)
    g = ma.embedding_backward(d, t, torch.empty(3, cols, device=DEV))
    for v in range(3):
        assert torch.equal(g[v], d[t == v].float().sum(0))


def test_most_norm_rows():
    rows = 1 << 24
    say("most norm rows")
    x = rand((rows, 3), 196, BF16)
    y, stats = ma.layernorm_forward(x)
    for part in (slice(0, 700), slice(rows - 700, rows)):
        ys, ss = ma.layernorm_forward(x[part].contiguous())
        assert torch.equal(y[part], ys) and torch.equal(stats[part], ss)
    db = torch.empty(3, device=DEV)
    dx = ma.layernorm_backward(torch.ones_like(x), x, stats, dbias=db)
    assert bool((db == rows).all()) and not dx.isnan().any()


@pytest.mark.parametrize("rows,cols", [(3, 1 << 24), (1 << 24, 1)])
@pytest.mark.parametrize("dt", [F32, BF16])
def test_largest_checkpoints(rows, cols, dt):
    say("largest checkpoints", rows, cols, dt)
    x = whole((rows, cols), 197, dt, 8)
    assert torch.equal(ma.act_unpack(ma.act_pack(x), dtype=dt), x)


@pytest.mark.parametrize("n,k", [(1 << 23, 1), (1, 1 << 23), (1 << 23, 200)])
@pytest.mark.parametrize("dyd", [F32, BF16])
def test_largest_weight_gradients(n, k, dyd):
    say("largest weight gradients", n, k, dyd)
    t = 70
    dy, x = whole((t, n), 198, dyd), whole((t, k), 199, BF16, 8)
    got = ma.act_weight_grad(dy, ma.act_pack(x), torch.empty(n, k, device=DEV))
    for part in (slice(0, 5000), slice(max(n, k) - 5000, None)):
        if n > k:
            assert torch.equal(got[part].double(), product(dy[:, part], x))
        else:
            assert torch.equal(got[:, part].double(), product(dy, x[:, part]))
