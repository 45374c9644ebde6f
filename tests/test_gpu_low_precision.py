"""GPU parity of root-mean-square norm, 4-bit matrices and their product against
the fp64 oracle (oracle/train_ops.py), and a run of them that ends in an optimizer
step.

Error bounds as in test_gpu_ops.py: u = 2^-24 is half an fp32 step; a sum of n fp32
terms in any order is off by at most n u times the sum of the magnitudes; a result
rounded once to type t by half a step more."""
import ctypes as C

import numpy as np
import pytest
import torch

import adamw_optimizer_step_amd as ma
from adamw_optimizer_step_amd import _lib as L
from gpu_util import need_gpu, say, to_np
from oracle import train_ops as T
from test_gpu_ops import BF16, DEPTH, DEV, F32, NORM_SHAPES, U, close, f64, guards, half, rand, view

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


# ---------------------------------------------------------------------------
# root-mean-square norm
# ---------------------------------------------------------------------------
def rms_inputs(rows, cols, xd, rd, seed):
    x = rand((rows, cols), seed, F32, 2.0) + rand((rows, 1), seed + 1, F32, 1.0)
    if rows > 2:
        x[1] = 0.0
    r = None if rd is None else rand((rows, cols), seed + 2, rd, 3.0)
    if r is not None and rows > 2:
        r[1] = 0.0
    return x.to(xd), r, 1 + rand((cols,), seed + 3, F32, 0.3)


def rms_y_tol(t, rstd, gain, y):
    """The sum of squares is off by depth u of itself, its mean and root by 4 u more (v_rsq_f32: a unit in the last
    place); then two products."""
    return np.abs(y) * (0.5 * (DEPTH + 4) * U + 4 * U + 2 * U)


@pytest.mark.parametrize("rows,cols", NORM_SHAPES)
@pytest.mark.parametrize("xd,rd,yd,gained,off", [(BF16, BF16, BF16, True, 0), (BF16, F32, BF16, True, 1), (F32, F32, F32, False, 3), (BF16, None, BF16, True, 1),
                                                 (F32, None, BF16, True, 0), (F32, BF16, F32, True, 0), (BF16, BF16, F32, False, 0)])
def test_rmsnorm_forward(rows, cols, xd, rd, yd, gained, off):
    say("rmsnorm_forward", rows, cols, xd, rd, yd, gained, off)
    x, r, gain = rms_inputs(rows, cols, xd, rd, 100)
    gain = gain if gained else None
    y, t, rstd = T.rmsnorm_forward(f64(x), None if gain is None else f64(gain), None if r is None else to_np(r), bf16_stream=rd == BF16)
    _, xv = view(x, off)
    rv = None if r is None else view(r, off)[1]
    yb, yv = view(torch.zeros(rows, cols, dtype=yd, device=DEV), off)
    tb, tv = (None, None) if r is None else view(torch.zeros(rows, cols, dtype=rd, device=DEV), off)
    ck = ma.ActCheckpoint.empty(rows, cols, DEV)
    out, total, got = ma.rmsnorm_forward(xv, gain, rv, out=yv, total=tv, held=ck)
    assert out is yv and total is (xv if r is None else tv)
    assert np.array_equal(f64(total), t)
    close(got, rstd[:, 0], rstd[:, 0] * (0.5 * (DEPTH + 4) + 4) * U)
    close(yv, y, rms_y_tol(t, rstd, gain, y), yd)
    assert guards(yb, rows * cols, off) and (r is None or guards(tb, rows * cols, off))
    # the same bits without the 8 bits, and however the operands are aligned (another type of y is another order of sums)
    y2, t2, rstd2 = ma.rmsnorm_forward(x, gain, r, dtype=yd)
    assert torch.equal(rstd2, got) and torch.equal(t2, total) and torch.equal(y2, yv)
    # the 8 bits are those of the fp32 y that the same call writes
    ck2 = ma.ActCheckpoint.empty(rows, cols, DEV)
    y32, _, _ = ma.rmsnorm_forward(x, gain, r, out=torch.empty(rows, cols, device=DEV), held=ck2)
    q, s = T.act_pack(f64(y32))
    assert np.array_equal(ck2.q.cpu().numpy(), q) and np.array_equal(ck2.scale.cpu().numpy(), s)
    # without y: those of the call that writes it in bf16
    h, t3, rstd3 = ma.rmsnorm_forward(x, gain, r, held=ck2)
    assert h is ck2 and torch.equal(t3, total)
    if yd == BF16:
        assert torch.equal(ck2.q, ck.q) and torch.equal(ck2.scale, ck.scale) and torch.equal(rstd3, got)


def test_rmsnorm_shapes_and_defaults():
    x = rand((2, 3, 40), 110, BF16)
    y, total, rstd = ma.rmsnorm_forward(x)
    assert y.shape == x.shape and y.dtype == BF16 and total is x and rstd.shape == (6,)
    y, total, rstd = ma.rmsnorm_forward(x, residual=x.float(), dtype=F32)
    assert y.dtype == F32 and total.dtype == F32 and total.shape == x.shape
    y, total, rstd = ma.rmsnorm_forward(x[:0], residual=x[:0])
    assert y.shape == total.shape == (0, 3, 40) and rstd.shape == (0,)
    dg = torch.ones(40, device=DEV)
    assert ma.rmsnorm_backward(y, total, rstd, dgain=dg, accumulate=True).shape == (0, 3, 40) and bool((dg == 1).all())
    ma.rmsnorm_backward(y, total, rstd, dgain=dg)
    assert not dg.any()


def test_rmsnorm_nonfinite_and_overflowing_rows_stay_in_their_row():
    x, r = rand((7, 700), 111), rand((7, 700), 112, BF16)
    x[2, 13], x[4, 699], x[5, 0] = float("nan"), float("inf"), 3e38
    ck = ma.ActCheckpoint.empty(7, 700, DEV)
    y, t, rstd = ma.rmsnorm_forward(x, residual=r, out=torch.empty_like(x), held=ck)
    assert torch.isnan(y[2]).all() and torch.isnan(y[4, 699]) and not y[4, :699].any()   # x / inf
    assert not y[5].any() and float(rstd[5]) == 0 and float(rstd[4]) == 0 and torch.isnan(rstd[2])
    ok = [0, 1, 3, 6]
    y2, t2, rstd2 = ma.rmsnorm_forward(x[ok].contiguous(), residual=r[ok].contiguous())
    assert torch.equal(y[ok], y2) and torch.equal(t[ok], t2) and torch.equal(rstd[ok], rstd2)
    # beyond the columns the checkpoint holds zeros in every row
    assert not ck.q[:, 700:].any()


@pytest.mark.parametrize("eps", [0.0, 1e-40, 1e-30])
def test_rmsnorm_of_zeros(eps):
    x = torch.zeros(3, 130, device=DEV)
    y, _, rstd = ma.rmsnorm_forward(x, eps=eps)
    if eps == 0.0:
        assert torch.isinf(rstd).all() and torch.isnan(y).all()
    else:
        want = 1.0 / np.sqrt(float(np.float32(eps)))
        close(rstd, np.full(3, want), 4 * U * want)
        assert not y.any()


def rms_dx_tol(dy, t, rstd, gain, dtotal):
    """g and xh are off by 2 u each, the mean by depth u; each of the two terms by 3 u more, the sum with dtotal by one."""
    xh, g = np.abs(t) * rstd, np.abs(dy) * (1.0 if gain is None else np.abs(gain))
    tol = rstd * (DEPTH + 12) * U * (g + xh * (g * xh).mean(1, keepdims=True))
    return tol if dtotal is None else tol + U * (np.abs(dtotal) + rstd * (g + xh * (g * xh).mean(1, keepdims=True)))


@pytest.mark.parametrize("rows,cols", NORM_SHAPES)
@pytest.mark.parametrize("kind,dyd,gained,stream,off", [("f32", F32, True, True, 0), ("bf16", BF16, True, True, 1), ("8", BF16, True, False, 0), ("8", F32, False, True, 1),
                                                        ("bf16", F32, True, False, 0), ("f32", BF16, False, True, 3)])
def test_rmsnorm_backward(rows, cols, kind, dyd, gained, stream, off):
    say("rmsnorm_backward", rows, cols, kind, dyd, gained, stream, off)
    t, _, gain = rms_inputs(rows, cols, F32 if kind == "f32" else BF16, None, 120)
    gain = gain if gained else None
    _, _, rstd = ma.rmsnorm_forward(t)
    dy = rand((rows, cols), 124, dyd, 0.1)
    tin, tn = t, f64(t)
    if kind == "8":
        tin = ma.act_pack(t)
        tn = T.act_unpack(*T.act_pack(tn), cols)
    else:
        _, tin = view(t, off)
    dxd = dyd if kind == "8" else t.dtype
    dt = rand((rows, cols), 125, dxd, 0.1) if stream else None
    dtv = view(dt, off)[1] if stream else None
    st, dtn, gn = f64(rstd)[:, None], None if dt is None else f64(dt), None if gain is None else f64(gain)
    dx, dgain = T.rmsnorm_backward(f64(dy), tn, st, gn, dtn)
    _, dyv = view(dy, off)
    db, dxv = view(torch.zeros(rows, cols, dtype=dxd, device=DEV), off)
    g0 = rand((cols,), 126)
    gg = g0.clone()
    ma.rmsnorm_backward(dyv, tin, rstd, gain, dtotal=dtv, dgain=gg, dx=dxv)
    close(dxv, dx, rms_dx_tol(f64(dy), tn, st, gn, dtn), dxd)
    assert guards(db, rows * cols, off)
    mag = (np.abs(f64(dy)) * np.abs(tn) * st).sum(0)   # a column's sum: every row one addition at most, products off by 3 u
    close(gg, dgain, (rows + 44) * U * mag)
    ag = g0.clone()
    dx2 = ma.rmsnorm_backward(dy, tin, rstd, gain, dtotal=dt, dgain=ag, accumulate=True)
    assert torch.equal(dx2, dxv) and torch.equal(ag, g0 + gg)
    assert torch.equal(ma.rmsnorm_backward(dy, tin, rstd, gain, dtotal=dt), dxv)


def test_rmsnorm_gradient_against_differences():
    """dx and dgain against central differences of the fp64 formula along random directions."""
    rows, cols = 4, 200
    x, r, gain = rms_inputs(rows, cols, F32, F32, 130)
    x[1] = rand((cols,), 134)
    dy, dt = rand((rows, cols), 135), rand((rows, cols), 136)
    _, t, rstd = ma.rmsnorm_forward(x, gain, r)
    dg = torch.empty(cols, device=DEV)
    dx = ma.rmsnorm_backward(dy, t, rstd, gain, dtotal=dt, dgain=dg)
    f = lambda t, g: (T.rmsnorm_forward(t, g)[0] * f64(dy)).sum() + (t * f64(dt)).sum()  # noqa: E731
    rng, h = np.random.default_rng(0), 1e-5
    base = [f64(t), f64(gain)]
    for k, grad in enumerate((dx, dg)):
        v = rng.standard_normal(base[k].shape)
        p, m = list(base), list(base)
        p[k], m[k] = base[k] + h * v, base[k] - h * v
        diff = (f(*p) - f(*m)) / (2 * h)
        # the kernel's gradient is off by its bound times |v|, as rstd itself is off by (depth / 2 + 6) u of the rest;
        # the quotient by the third derivative's h^2 / 6, some 1e-10 of |y dy|, and by the rounding of f over h
        st = f64(rstd)[:, None]
        own = [rms_dx_tol(f64(dy), f64(t), st, f64(gain), f64(dt)) * 2, (rows + 44 + DEPTH) * U * np.abs(f64(dy) * 6.0).sum(0)][k]   # |xh| < 6 here
        mag = np.abs(T.rmsnorm_forward(*base)[0] * f64(dy)).sum() + np.abs(f64(t) * f64(dt)).sum()
        assert abs(diff - (f64(grad) * v).sum()) <= (own * np.abs(v)).sum() + (2.0 ** -52 / h * 16 + 1e-8) * mag


# ---------------------------------------------------------------------------
# 4-bit matrices
# ---------------------------------------------------------------------------
def wild(rows, cols, dt, seed):
    """Rows of every magnitude, zeros, blocks with NaN and infinities, the largest value."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((rows, cols)) * 2.0 ** rng.integers(-140, 126, (rows, 1))
    x[rng.random((rows, cols)) < 0.1] = 0.0
    x.flat[::97] *= -2.0 ** -20
    x = torch.from_numpy(x).float().to(dt)
    if rows > 2:
        x[1] = 0
        x[2, 0], x[2, -1], x[2, cols // 2] = float("inf"), float("-inf"), float("nan")
        x[0, 0] = torch.finfo(dt).max
    return x.to(DEV)


MX_SHAPES = [(1, 1), (3, 7), (2, 128), (5, 129), (17, 1000), (64, 1024), (3, 4099), (257, 136), (130, 31), (300, 2), (33, 65), (255, 8), (1, 200)]


@pytest.mark.parametrize("rows,cols", MX_SHAPES)
@pytest.mark.parametrize("dt,off", [(F32, 0), (BF16, 0), (BF16, 1), (F32, 3)])
@pytest.mark.parametrize("transpose", [False, True])
def test_mx4_bits(rows, cols, dt, off, transpose):
    say("mx4", rows, cols, dt, off, transpose)
    x = wild(rows, cols, dt, rows * cols)
    xb, xv = view(x, off)
    src = f64(x).T if transpose else f64(x)
    m = ma.mx4_pack(xv, transpose=transpose)
    q, s = T.mx4_pack(src)
    assert (m.rows, m.cols) == src.shape
    assert np.array_equal(m.scale.cpu().numpy(), s)
    assert np.array_equal(m.q.cpu().numpy(), q)
    want = T.mx4_unpack(q, s, src.shape[1]).astype(np.float32)
    for od in (F32, BF16):
        ob, ov = view(torch.zeros(src.shape, dtype=od, device=DEV), off)
        ma.mx4_unpack(m, out=ov)
        assert np.array_equal(to_np(ov), want, equal_nan=True) and guards(ob, src.size, off)
    assert guards(xb, rows * cols, off)
    # into buffers of the caller's, the scales apart
    n = ma.Mx4Matrix(torch.full_like(m.q, 9), torch.full_like(m.scale, 9), m.cols)
    assert ma.mx4_pack(xv, transpose=transpose, out=n) is n and torch.equal(n.q, m.q) and torch.equal(n.scale, m.scale)


@pytest.mark.parametrize("transpose", [False, True])
def test_mx4_rounds_every_bf16_value_as_defined(transpose):
    """All 65536 bf16 patterns, each beside every magnitude class of block maximum."""
    v = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(BF16).view(2048, 32)
    finite = torch.isfinite(v.float())
    v = torch.where(finite, v, torch.zeros_like(v))
    for k in range(0, 255, 5):
        top = torch.tensor([k << 7 | 0x5F], dtype=torch.int32).to(torch.int16).view(BF16)
        x = v.clone()
        x[:, 0] = top
        x = torch.where(x.float().abs() <= top.float().abs(), x, torch.zeros_like(x))
        src = x.view(512, 128)
        m = ma.mx4_pack(src.t().contiguous().to(DEV), transpose=True) if transpose else ma.mx4_pack(src.to(DEV))
        q, s = T.mx4_pack(f64(src))
        assert np.array_equal(m.q.cpu().numpy(), q) and np.array_equal(m.scale.cpu().numpy(), s), k


def test_mx4_unpacks_every_byte():
    q = torch.arange(256, dtype=torch.uint8).repeat(64, 1)[:, :64].contiguous()
    q = torch.cat([q, q + 64, q + 128, q + 192]).to(DEV)
    s = torch.arange(256, dtype=torch.uint8).view(1, 256, 1).expand(1, 256, 4).contiguous().to(DEV)
    got = ma.mx4_unpack(ma.Mx4Matrix(q, s, 128), dtype=F32)
    with np.errstate(over="ignore"):
        assert np.array_equal(to_np(got), T.mx4_unpack(q.cpu().numpy(), s.cpu().numpy(), 128).astype(np.float32), equal_nan=True)


def test_mx4_of_views_and_batches():
    x = rand((3, 5, 40), 140, BF16)
    m = ma.mx4_pack(x)
    assert (m.rows, m.cols) == (15, 40) and ma.mx4_unpack(m).shape == (15, 40)
    out = torch.empty(3, 5, 40, device=DEV)
    assert ma.mx4_unpack(m, out=out) is out and torch.equal(out.view(15, 40), ma.mx4_unpack(m, dtype=F32))
    assert (lambda e: (e.rows, e.q.shape[0]))(ma.mx4_pack(x[:0])) == (0, 0)
    t = ma.mx4_pack(x, transpose=True)
    assert torch.equal(ma.mx4_unpack(t), ma.mx4_unpack(ma.mx4_pack(x.view(15, 40).t().contiguous())))


# ---------------------------------------------------------------------------
# the product
# ---------------------------------------------------------------------------
def held(rows, cols, bits, seed, scale=1.0):
    """A held matrix and its values in fp64."""
    x = rand((rows, cols), seed, BF16, scale) * torch.exp2(torch.randint(-3, 4, (rows, 1), generator=torch.Generator().manual_seed(seed + 1)).float()).to(DEV)
    m = ma.mx4_pack(x.bfloat16()) if bits == 4 else ma.act_pack(x.bfloat16())
    return m, f64(ma.mx4_unpack(m, dtype=F32) if bits == 4 else ma.act_unpack(m, dtype=F32))


def product_tol(mag, ins):
    """Products of held values are exact; each of the padded k is one addition at most, off by a whole unit (2 u) where
    the matrix instruction cuts off, and the shares of a split one more each."""
    return (-(-ins // 128) * 128 + 64) * 2 * U * mag


PRODUCTS = [(1, 1, 1), (1, 16, 128), (3, 5, 7), (16, 33, 130), (17, 64, 300), (33, 100, 127), (64, 65, 1000), (1, 1003, 4099), (129, 250, 333), (100, 16, 64),
            (128, 128, 128), (130, 129, 257), (255, 300, 640), (257, 513, 129), (300, 1030, 1500), (31, 2050, 2000), (5, 7, 9000), (1030, 70, 260), (520, 515, 513),
            (1, 8200, 520), (48, 48, 4200), (700, 260, 8321)]


@pytest.mark.parametrize("rows,outs,ins", PRODUCTS)
@pytest.mark.parametrize("bits,yd,acc,off", [(4, BF16, False, 0), (4, F32, True, 1), (8, BF16, True, 3), (8, F32, False, 0), (4, F32, False, 3), (8, BF16, False, 1)])
def test_product(rows, outs, ins, bits, yd, acc, off):
    say("mx4_matmul", rows, outs, ins, bits, yd, acc, off)
    x, xn = held(rows, ins, bits, 150)
    w, wn = held(outs, ins, 4, 152, 0.05)
    y0 = rand((rows, outs), 154, yd)
    want, mag = T.mx4_matmul(xn, wn, f64(y0) if acc else None)
    yb, yv = view(y0, off)
    assert ma.mx4_matmul(x, w, out=yv, accumulate=acc) is yv
    close(yv, want, product_tol(mag, ins) + (U * (np.abs(f64(y0)) + mag) if acc else 0), yd)
    assert guards(yb, rows * outs, off)
    again = y0.clone()
    ma.mx4_matmul(x, w, out=again, accumulate=acc)
    assert torch.equal(again, yv)   # the same bits, however y is aligned


@pytest.mark.parametrize("rows,outs,ins", [(1, 40, 300), (16, 200, 1000), (20, 64, 4000), (65, 64, 700), (200, 300, 1030), (520, 770, 390), (1100, 1300, 260)])
@pytest.mark.parametrize("bits", [4, 8])
def test_product_of_whole_numbers_is_exact(rows, outs, ins, bits):
    """Sums of products of small whole numbers are below 2^24: every order of exact additions gives the same bits. The
    values differ along both axes, so that a product put in another's place shows."""
    say("mx4_matmul, whole numbers", rows, outs, ins, bits)
    g = torch.Generator().manual_seed(160)
    table = torch.tensor([0, 1, 2, 3, 4, 6, -1, -2, -3, -4, -6], dtype=F32)
    xv, wv = (table[torch.randint(0, 11, (n, ins), generator=g)] for n in (rows, outs))
    xv[:, ::32], wv[:, ::32] = 6, -6      # every block's exponent 0
    x = xv.to(DEV)
    x = ma.mx4_pack(x) if bits == 4 else ma.act_pack(x)
    w = ma.mx4_pack(wv.to(DEV))
    assert torch.equal(ma.mx4_unpack(w, dtype=F32).cpu(), wv)
    got = ma.mx4_matmul(x, w, dtype=F32)
    assert np.array_equal(f64(got), xv.double().numpy() @ wv.double().numpy().T)
    got = ma.mx4_matmul(x, w, out=torch.full((rows, outs), 5.0, device=DEV), accumulate=True)
    assert np.array_equal(f64(got), xv.double().numpy() @ wv.double().numpy().T + 5)


@pytest.mark.parametrize("rows", [1, 40, 300])
@pytest.mark.parametrize("bits", [4, 8])
def test_product_takes_every_scale(rows, bits):
    """Each block of 32 has its own power of two, over the whole range; products beyond fp32 are infinite, below it zero."""
    g = torch.Generator().manual_seed(170)
    outs, ins = 70, 512
    e = torch.randint(1, 253, (ins // 128, outs, 4), generator=g).to(torch.uint8)
    wq = torch.full((outs, ins // 2), 0x22, dtype=torch.uint8)      # ones
    w = ma.Mx4Matrix(wq.to(DEV), e.to(DEV), ins)
    ex = torch.randint(90, 160, (rows, ins // 128) if bits == 8 else (ins // 128, rows, 4), generator=g).to(torch.uint8)
    one = 0x38 if bits == 8 else 0x22
    xq = torch.full((rows, ins if bits == 8 else ins // 2), one, dtype=torch.uint8)
    x = (ma.ActCheckpoint if bits == 8 else ma.Mx4Matrix)(xq.to(DEV), ex.to(DEV), ins)
    xn = T.act_unpack(xq.numpy(), ex.numpy(), ins) if bits == 8 else T.mx4_unpack(xq.numpy(), ex.numpy(), ins)
    wn = T.mx4_unpack(wq.numpy(), e.numpy(), ins)
    want = xn @ wn.T
    got = f64(ma.mx4_matmul(x, w, dtype=F32))
    # sums of positive terms: off by ins 2 u of the result; a sum near fp32's largest may pass it
    edge = np.abs(want) > 2.0 ** 127.9
    assert np.all(np.isinf(got[want > 2.0 ** 129]))
    ok = ~edge
    assert np.all(np.abs(got - want)[ok] <= ins * 2 * U * want[ok] + 2.0 ** -126)


@pytest.mark.parametrize("rows", [5, 70, 300])
@pytest.mark.parametrize("bits", [4, 8])
def test_product_keeps_nonfinite_values_in_their_row_and_column(rows, bits):
    outs, ins = 300, 700
    xv, wv = rand((rows, ins), 180, BF16), rand((outs, ins), 181, BF16)
    xv[3, 600], wv[7, 5], wv[299, 699] = float("nan"), float("inf"), float("nan")
    x = ma.mx4_pack(xv) if bits == 4 else ma.act_pack(xv)
    got = ma.mx4_matmul(x, ma.mx4_pack(wv), dtype=F32)
    bad = torch.zeros(rows, outs, dtype=torch.bool, device=DEV)
    bad[3], bad[:, 7], bad[:, 299] = True, True, True
    assert torch.equal(torch.isnan(got), bad) and bool(torch.isfinite(got[~bad]).all())


def plan(rows, outs, ins, bits):
    e, n = C.c_int32(-1), C.c_int32(-1)
    assert L.lib().ma_test_mx4_matmul_plan(rows, outs, ins, bits, C.byref(e), C.byref(n)) == 0
    return e.value, n.value


# (sizes, the output tile's edge, whether the columns are split, whether a block works on several tiles): every form,
# k-tiles fewer than are kept ahead and more, ragged edges, several tiles after one another
FORMS = [(1300, 1700, 900, 128, False, False), (2100, 2100, 300, 128, False, False), (5000, 5003, 100, 128, False, True), (9001, 4100, 260, 128, False, True),
         (4400, 2101, 390, 128, False, True), (900, 521, 20000, 128, True, False), (300, 700, 16000, 128, True, False), (6000, 9001, 700, 256, False, True),
         (2000, 2050, 9000, 256, True, False), (2049, 2047, 12000, 256, True, False), (7000, 7101, 1900, 256, False, True), (4401, 1857, 16761, 256, True, True)]


@pytest.mark.parametrize("rows,outs,ins,edge,split,several", FORMS)
@pytest.mark.parametrize("bits,yd,acc,off", [(4, BF16, False, 1), (4, F32, True, 3), (8, BF16, True, 0), (8, F32, False, 1)])
def test_product_of_every_form(rows, outs, ins, edge, split, several, bits, yd, acc, off):
    say("mx4_matmul form", rows, outs, ins, edge, split, several, bits, yd, acc, off)
    e, n = plan(rows, outs, ins, bits)
    jobs = -(-rows // e) * -(-outs // e) * n
    assert (e, n > 1, jobs > (512 if e == 128 else 256)) == (edge, split, several)
    g = torch.Generator(device=DEV).manual_seed(155)
    x = torch.randn(rows, ins, generator=g, device=DEV) * torch.exp2(torch.randint(-3, 4, (rows, 1), generator=g, device=DEV).float())
    w = ma.mx4_pack(torch.randn(outs, ins, generator=g, device=DEV) * 0.05)
    x = ma.mx4_pack(x) if bits == 4 else ma.act_pack(x)
    xn = (ma.mx4_unpack(x, dtype=F32) if bits == 4 else ma.act_unpack(x, dtype=F32)).double()
    wn = ma.mx4_unpack(w, dtype=F32).double()
    y0 = torch.randn(rows, outs, generator=g, device=DEV).to(yd)
    want, mag = torch.mm(xn, wn.t()), torch.mm(xn.abs(), wn.abs().t())
    yb, yv = view(y0, off)
    ma.mx4_matmul(x, w, out=yv, accumulate=acc)
    tol = product_tol(mag, ins)
    if acc:
        want, tol = want + y0.double(), tol + U * (y0.double().abs() + mag)
    bound = tol * (1 + half(yd)) + half(yd) * want.abs() + 2.0 ** -126
    assert bool(((yv.double() - want).abs() <= bound).all())
    assert guards(yb, rows * outs, off)
    again = y0.clone()
    ma.mx4_matmul(x, w, out=again, accumulate=acc)
    assert torch.equal(again, yv)


@pytest.mark.parametrize("rows,outs,ins", [f[:3] for f in FORMS])
@pytest.mark.parametrize("bits", [4, 8])
def test_product_of_whole_numbers_is_exact_in_every_form(rows, outs, ins, bits):
    say("mx4_matmul form, whole numbers", rows, outs, ins, bits)
    g = torch.Generator(device=DEV).manual_seed(165)
    table = torch.tensor([0, 1, 2, 3, 4, 6, -1, -2, -3, -4, -6], dtype=F32, device=DEV)
    xv, wv = (table[torch.randint(0, 11, (n, ins), generator=g, device=DEV)] for n in (rows, outs))
    xv[:, ::32], wv[:, ::32] = 6, -6      # every block's exponent 0
    w = ma.mx4_pack(wv)
    x = ma.mx4_pack(xv) if bits == 4 else ma.act_pack(xv)
    want = torch.mm(xv.double(), wv.double().t())
    assert torch.equal(ma.mx4_matmul(x, w, dtype=F32).double(), want)
    assert torch.equal(ma.mx4_matmul(x, w, out=torch.full((rows, outs), 5.0, device=DEV), accumulate=True).double(), want + 5)


@pytest.mark.parametrize("rows,outs,ins", [(1300, 1700, 900), (900, 521, 20000), (3000, 6001, 700), (2000, 2050, 9000)])
@pytest.mark.parametrize("bits", [4, 8])
def test_product_keeps_nonfinite_values_apart_in_every_form(rows, outs, ins, bits):
    g = torch.Generator(device=DEV).manual_seed(175)
    xv, wv = (torch.randn(n, ins, generator=g, device=DEV) for n in (rows, outs))
    xv[rows - 1, ins - 1], xv[130, 0], wv[7, 5], wv[outs - 1, ins - 1] = float("nan"), float("nan"), float("inf"), float("nan")
    x = ma.mx4_pack(xv) if bits == 4 else ma.act_pack(xv)
    got = ma.mx4_matmul(x, ma.mx4_pack(wv))
    bad = torch.zeros(rows, outs, dtype=torch.bool, device=DEV)
    bad[rows - 1], bad[130], bad[:, 7], bad[:, outs - 1] = True, True, True, True
    assert torch.equal(torch.isnan(got), bad) and bool(torch.isfinite(got[~bad]).all())


def beside_large(rows, outs, ins):
    """8-bit rows whose small values stand beside large ones in every 8 of them, and weights: all products are multiples of
    2^-10, and only three columns of the largest values have weights, so that sums stay below 2^14."""
    g = torch.Generator(device=DEV).manual_seed(181)
    xv = torch.randint(-15, 16, (rows, ins), generator=g, device=DEV).float() * 2.0 ** -9
    middle = torch.randint(-15, 16, (rows, ins), generator=g, device=DEV).float() * 2.0 ** -2
    xv = torch.where(torch.rand(rows, ins, generator=g, device=DEV) < 0.1, middle, xv)
    table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.5, -1, -1.5, -2, -3, -4, -6], device=DEV)
    wv = table[torch.randint(0, 15, (outs, ins), generator=g, device=DEV)]
    wv[:, ::32] = 6                                        # every block's exponent 0
    at = torch.arange(0, ins, 128, device=DEV)
    large = torch.minimum(at + at // 128 * 37 % 128, torch.tensor(ins - 1, device=DEV))
    xv[:, large] = 448.0 * (1 - 2 * torch.randint(0, 2, (rows, large.numel()), generator=g, device=DEV).float())
    wv[:, large] = 0
    wv[:, large[::max(1, large.numel() // 3)][:3]] = 4
    x, w = ma.act_pack(xv), ma.mx4_pack(wv)
    assert torch.equal(ma.act_unpack(x, dtype=F32), xv) and torch.equal(ma.mx4_unpack(w, dtype=F32), wv)
    return x, w, xv.double(), wv.double()


@pytest.mark.parametrize("rows,outs,ins", [(1, 40, 300), (3, 17, 100), (20, 64, 4000), (60, 64, 700), (200, 300, 1030)] + [f[:3] for f in FORMS])
def test_product_of_8_bit_rows_keeps_small_products_beside_large_ones(rows, outs, ins):
    """All sums are whole multiples of 2^-10 below 2^14: fp32 results have every bit. A bf16 result may lose, of 7
    products of 8, less than 2^-13 of the largest one's power of two, beside its own rounding."""
    say("mx4_matmul, small beside large", rows, outs, ins)
    x, w, xv, wv = beside_large(rows, outs, ins)
    want = torch.mm(xv, wv.t())
    assert torch.equal(ma.mx4_matmul(x, w, dtype=F32).double(), want)
    assert torch.equal(ma.mx4_matmul(x, w, out=torch.full((rows, outs), 0.25, device=DEV), accumulate=True).double(), want + 0.25)
    pad = torch.nn.functional.pad
    most = torch.mm(pad(xv, (0, -ins % 8)).abs().view(rows, -1, 8).amax(2), pad(wv, (0, -ins % 8)).abs().view(outs, -1, 8).amax(2).t())
    got = ma.mx4_matmul(x, w).double()
    cut = 7 * 2.0 ** -13 * most + product_tol(torch.mm(xv.abs(), wv.abs().t()), ins)
    assert bool(((got - want).abs() <= cut * (1 + half(BF16)) + half(BF16) * want.abs()).all())


@pytest.mark.parametrize("rows,outs", [(256, 256), (20, 256), (700, 900)])
@pytest.mark.parametrize("yd", [BF16, F32])
def test_product_takes_every_8_bit_value(rows, outs, yd):
    """Row r holds the byte r % 256 in column r % 256, and w is the identity; a NaN reaches its whole row."""
    say("mx4_matmul, every byte", rows, outs, yd)
    r = torch.arange(rows, device=DEV)
    q = torch.zeros(rows, 256, dtype=torch.uint8, device=DEV)
    q[r, r % 256] = (r % 256).to(torch.uint8)
    x = ma.ActCheckpoint(q, torch.full((rows, 2), 127 + 3, dtype=torch.uint8, device=DEV), 256)
    w = ma.mx4_pack(torch.eye(outs, 256, device=DEV))
    value = torch.arange(256, device=DEV).to(torch.uint8).view(torch.float8_e4m3fn).float() * 8
    want = torch.zeros(rows, outs, device=DEV)
    want[r, r % 256] = value[r % 256]
    want[torch.isnan(value[r % 256])] = float("nan")
    got = ma.mx4_matmul(x, w, dtype=yd)
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(torch.nan_to_num(got.float()), torch.nan_to_num(want))


def test_product_shapes_and_defaults():
    x, w = ma.mx4_pack(rand((4, 40), 190)), ma.mx4_pack(rand((6, 40), 191))
    y = ma.mx4_matmul(x, w)
    assert y.shape == (4, 6) and y.dtype == BF16
    out = torch.empty(2, 2, 6, device=DEV)
    assert ma.mx4_matmul(x, w, out=out) is out and torch.equal(out.view(4, 6), ma.mx4_matmul(x, w, dtype=F32))
    assert ma.mx4_matmul(ma.mx4_pack(torch.empty(0, 40, device=DEV)), w).shape == (0, 6)


@pytest.mark.parametrize("rows,outs,ins", [(7, 48, 200), (300, 200, 1000)])
def test_product_is_bilinear(rows, outs, ins):
    """<x w^T, d> = <w, d^T x> = <x, d w>: the two gradients of a linear layer are products of the same kind."""
    x, xn = held(rows, ins, 4, 200)
    w, wn = held(outs, ins, 4, 202)
    y = f64(ma.mx4_matmul(x, w, dtype=F32))
    d, dn = held(rows, outs, 4, 204)
    wt, xt, dt = (ma.mx4_pack(torch.from_numpy(v).float().to(DEV), transpose=True) for v in (wn, xn, dn))
    dx, dw = f64(ma.mx4_matmul(d, wt, dtype=F32)), f64(ma.mx4_matmul(dt, xt, dtype=F32))
    wt, xt, dt = (f64(ma.mx4_unpack(v, dtype=F32)) for v in (wt, xt, dt))
    mag = np.abs(xn) @ np.abs(wn).T
    assert np.all(np.abs(y - xn @ wn.T) <= product_tol(mag, ins))
    assert np.all(np.abs(dx - dn @ wt.T) <= product_tol(np.abs(dn) @ np.abs(wt).T, outs))
    assert np.all(np.abs(dw - dt @ xt.T) <= product_tol(np.abs(dt) @ np.abs(xt).T, rows))


# ---------------------------------------------------------------------------
# streams, graphs, workspaces, a run of them
# ---------------------------------------------------------------------------
def sequence(s, stream=None, ws=None):
    """Norm to 8 bits, product, its gradient by 4-bit products and the 8-bit weight gradient, the norm's backward pass."""
    rows, cols = s["x"].shape
    heldy = s.get("held") or ma.ActCheckpoint.empty(rows, cols, DEV)
    _, total, rstd = ma.rmsnorm_forward(s["x"], s["gain"], s["res"], held=heldy, stream=stream)
    w4, wt4 = ma.mx4_pack(s["w"], stream=stream), ma.mx4_pack(s["w"], transpose=True, stream=stream)
    out = ma.mx4_matmul(heldy, w4, stream=stream)
    d4 = ma.mx4_pack(s["dout"], stream=stream)
    dy = ma.mx4_matmul(d4, wt4, stream=stream)
    dw = ma.act_weight_grad(s["dout"], heldy, torch.empty_like(s["w"]), stream=stream)
    dgain = torch.empty_like(s["gain"])
    dx = ma.rmsnorm_backward(dy, total, rstd, s["gain"], dtotal=s["dtotal"], dgain=dgain, stream=stream)
    return [total, rstd, out, dy, dw, dgain, dx]


def sequence_state(rows, cols, outs, seed):
    return dict(x=rand((rows, cols), seed, BF16), res=rand((rows, cols), seed + 1, BF16), gain=1 + rand((cols,), seed + 2, F32, 0.1),
                w=rand((outs, cols), seed + 3, BF16, 0.05), dout=rand((rows, outs), seed + 4, BF16, 0.01), dtotal=rand((rows, cols), seed + 5, BF16, 0.01))


@pytest.mark.parametrize("rows,cols,outs", [(3, 130, 70), (70, 500, 260), (1300, 260, 520)])
def test_other_streams_give_the_same_bits(rows, cols, outs):
    s = sequence_state(rows, cols, outs, 210)
    want = sequence(s)
    torch.cuda.synchronize()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    for st in (a, b):
        st.wait_stream(torch.cuda.current_stream())
    got = [sequence(s, stream=st) for st in (a, b)]          # two sequences at once
    with torch.cuda.stream(a):
        got.append(sequence(s))
    torch.cuda.synchronize()
    for g in got:
        assert all(torch.equal(p, q) for p, q in zip(g, want))


@pytest.mark.parametrize("rows,cols,outs", [(1, 256, 300), (70, 500, 260), (1300, 260, 520)])
def test_graph_replays_give_the_eager_bits(rows, cols, outs):
    s = sequence_state(rows, cols, outs, 220)
    sequence(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = sequence(s)
    for k in range(3):
        n = sequence_state(rows, cols, outs, 230 + 10 * k)
        for name in s:
            s[name].copy_(n[name])
        graph.replay()
        torch.cuda.synchronize()
        want = sequence(s)      # eager work between the replays
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, want))


def test_two_products_at_once_with_workspaces_of_their_own():
    cases = [(300, 200, 9000, 4), (70, 130, 5000, 8)]
    sets = [(held(r, k, b, 250)[0], held(n, k, 4, 252)[0], ma.mx4_matmul_workspace_size(r, n, k, b)) for r, n, k, b in cases]
    want = [ma.mx4_matmul(x, w, dtype=F32) for x, w, _ in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    ws = [torch.full((max(n, 1) + 512,), 255, dtype=torch.uint8, device=DEV) for _, _, n in sets]
    torch.cuda.synchronize()
    for _ in range(5):
        got = [ma.mx4_matmul(x, w, dtype=F32, workspace=ws[i], stream=streams[i]) for i, (x, w, n) in enumerate(sets)]
    torch.cuda.synchronize()
    for i, (g, y) in enumerate(zip(got, want)):
        assert torch.equal(g, y) and bool((ws[i][sets[i][2]:] == 255).all())


def test_training_step_of_a_low_precision_layer():
    """The run against the oracle: norm to 8 bits, product, backward, then Muon on the weights and AdamW on the gain."""
    rows, cols, outs = 200, 384, 256
    s = sequence_state(rows, cols, outs, 260)
    total, rstd, out, dy, dw, dgain, dx = sequence(s)
    y, t, r = T.rmsnorm_forward(f64(s["x"]), f64(s["gain"]), to_np(s["res"]), bf16_stream=True)
    assert np.array_equal(f64(total), t)
    y32, _, _ = ma.rmsnorm_forward(s["x"], s["gain"], s["res"], dtype=F32)
    close(y32, y, rms_y_tol(t, r, None, y))
    # y in 8 bits: off by half a step of e4m3, or of the block's least; the rest is checked on what is held
    h, _, _ = ma.rmsnorm_forward(s["x"], s["gain"], s["res"], held=ma.ActCheckpoint.empty(rows, cols, DEV))
    held8 = f64(ma.act_unpack(h, dtype=F32))
    amax = np.abs(held8).reshape(rows, -1, 128).max(-1, keepdims=True).repeat(128, 2).reshape(rows, cols)
    assert np.all(np.abs(held8 - y) <= np.maximum(2.0 ** -4 * np.abs(y), 2.0 ** -18 * 2 * amax) * (1 + 1e-5))
    w4, wt4 = (T.mx4_unpack(*T.mx4_pack(v), v.shape[1]) for v in (f64(s["w"]), f64(s["w"]).T))
    want, mag = T.mx4_matmul(held8, w4)
    close(out, want, product_tol(mag, cols), BF16)
    d4 = T.mx4_unpack(*T.mx4_pack(f64(s["dout"])), outs)
    want, mag = T.mx4_matmul(d4, wt4)
    close(dy, want, product_tol(mag, outs), BF16)
    want, mag = T.act_weight_grad(f64(s["dout"]), held8)
    close(dw, want, (rows + 100) * U * mag, BF16)
    wx, wg = T.rmsnorm_backward(f64(dy), t, f64(rstd)[:, None], f64(s["gain"]), f64(s["dtotal"]))
    close(dx, wx, rms_dx_tol(f64(dy), t, f64(rstd)[:, None], f64(s["gain"]), f64(s["dtotal"])), BF16)
    close(dgain, wg, (rows + 44) * U * (np.abs(f64(dy)) * np.abs(t) * r).sum(0) * (1 + 1e-5))
    w, g, m = s["w"][None], dw[None], torch.zeros_like(s["w"])[None]
    before, gain = w.clone(), s["gain"].clone()
    ma.muon_step([ma.MuonGroup(w, g, m)], ma.MuonHParams(lr=0.02, momentum=0.95, ns_steps=5, coeffs=ma.KELLER_JORDAN))
    z = torch.zeros_like(gain)
    ma.adamw_step([dict(param=gain, grad=dgain, exp_avg=z, exp_avg_sq=z.clone(), step=1, lr=1e-3, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.0)])
    torch.cuda.synchronize()
    assert bool(torch.isfinite(w).all()) and not torch.equal(w, before) and not torch.equal(gain, s["gain"])


# ---------------------------------------------------------------------------
# large operands
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("bits", [4, 8])
def test_product_of_operands_of_more_than_2_32_bytes(bits):
    """Rows far into x, and outputs far into y: the last rows are those of a call on them alone."""
    rows, outs, ins = (1 << 21) + 77, 600, 8200 if bits == 4 else 4100
    p = -(-ins // 128) * 128
    say("large product", rows, outs, ins, bits, rows * p * bits // 8)
    g = torch.Generator(device=DEV).manual_seed(270)
    if bits == 4:
        xq = torch.randint(0, 256, (rows, p // 2), generator=g, device=DEV, dtype=torch.uint8)
        xs = torch.randint(120, 130, (p // 128, rows, 4), generator=g, device=DEV, dtype=torch.uint8)
        x = ma.Mx4Matrix(xq, xs, ins)
        part = lambda a, b: ma.Mx4Matrix(xq[a:b].contiguous(), xs[:, a:b].contiguous(), ins)  # noqa: E731
    else:
        xq = torch.randint(0, 120, (rows, p), generator=g, device=DEV, dtype=torch.uint8)
        xs = torch.randint(120, 130, (rows, p // 128), generator=g, device=DEV, dtype=torch.uint8)
        x = ma.ActCheckpoint(xq, xs, ins)
        part = lambda a, b: ma.ActCheckpoint(xq[a:b].contiguous(), xs[a:b].contiguous(), ins)  # noqa: E731
    w = ma.mx4_pack(rand((outs, ins), 271, BF16))
    y = ma.mx4_matmul(x, w, dtype=F32)
    assert y.numel() * 4 > 1 << 32
    for a, b in ((0, 300), (rows - 300, rows), (rows // 2, rows // 2 + 300)):
        small = part(a, b)
        xn = f64(ma.mx4_unpack(small, dtype=F32) if bits == 4 else ma.act_unpack(small, dtype=F32))
        want, mag = T.mx4_matmul(xn, f64(ma.mx4_unpack(w, dtype=F32)))
        close(y[a:b], want, product_tol(mag, ins))


@pytest.mark.parametrize("transpose", [False, True])
def test_mx4_of_more_than_2_32_bytes(transpose):
    rows, cols = (1 << 20) + 33, 2050
    say("large mx4", rows, cols, transpose)
    x = torch.randn(rows, cols, generator=torch.Generator(device=DEV).manual_seed(280), device=DEV, dtype=F32)
    m = ma.mx4_pack(x, transpose=transpose)
    out = ma.mx4_unpack(m, dtype=F32)
    for a, b in ((0, 64), (rows - 33, rows), (rows // 2 // 32 * 32, rows // 2 // 32 * 32 + 96)):
        part = x[a:b]
        want = T.mx4_unpack(*T.mx4_pack(f64(part).T), part.shape[0]) if transpose else T.mx4_unpack(*T.mx4_pack(f64(part)), cols)
        got = out[:, a:b] if transpose else out[a:b]
        assert np.array_equal(to_np(got), want.astype(np.float32))


def test_rmsnorm_of_more_than_2_32_bytes():
    rows, cols = (1 << 20) + 5, 2055
    say("large rmsnorm", rows, cols)
    g = torch.Generator(device=DEV).manual_seed(290)
    x, r = (torch.randn(rows, cols, generator=g, device=DEV, dtype=F32).bfloat16() for _ in range(2))
    assert x.numel() * 2 > 1 << 32
    y, t, rstd = ma.rmsnorm_forward(x, residual=r)
    dg = torch.empty(cols, device=DEV)
    dx = ma.rmsnorm_backward(y, t, rstd, dtotal=x, dgain=dg)
    for a, b in ((0, 40), (rows - 40, rows)):
        y2, t2, s2 = ma.rmsnorm_forward(x[a:b].contiguous(), residual=r[a:b].contiguous())
        assert torch.equal(t[a:b], t2)
        close(y[a:b], f64(t2) * f64(s2)[:, None], rms_y_tol(None, None, None, f64(y2)), BF16)
        dn, _ = T.rmsnorm_backward(f64(y[a:b]), f64(t2), f64(rstd[a:b])[:, None], None, f64(x[a:b]))
        close(dx[a:b], dn, rms_dx_tol(f64(y[a:b]), f64(t2), f64(rstd[a:b])[:, None], None, f64(x[a:b])), BF16)
