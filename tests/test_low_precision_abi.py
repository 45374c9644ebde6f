"""Root-mean-square norm, 4-bit matrices and their product without a GPU: every
entry point rejects bad arguments before any launch, and the binding rejects
wrong types, shapes, strides and host tensors."""
import ctypes as C
import os

import pytest
import torch

import adamw_optimizer_step_amd as ma
from adamw_optimizer_step_amd import _lib as L

pytestmark = pytest.mark.skipif(not os.path.exists(L.LIB_PATH), reason="library not built")

BASE, GAP = 1 << 40, 1 << 36   # fake, never dereferenced device addresses
at = lambda i: BASE + i * GAP  # noqa: E731

CALLS = {
    "ma_rmsnorm_forward": dict(x=at(0), x_dtype=1, residual=at(1), residual_dtype=0, rows=10, cols=64, gain=at(2), eps=1e-5, total=at(3),
                               y=at(4), y_dtype=1, rstd=at(5), held_q=at(6), held_scale=at(7), stream=None),
    "ma_rmsnorm_backward": dict(dy=at(0), dy_dtype=1, t=at(1), t_dtype=1, held_q=None, held_scale=None, rows=10, cols=64, rstd=at(2),
                                gain=at(3), dtotal=at(4), dx=at(5), dx_dtype=1, dgain=at(6), accumulate=0, workspace=at(7),
                                workspace_bytes=1 << 30, stream=None),
    "ma_mx4_pack": dict(x=at(0), x_dtype=1, rows=10, cols=64, transpose=0, q=at(1), scale=at(2), stream=None),
    "ma_mx4_unpack": dict(q=at(0), scale=at(1), rows=10, cols=64, out=at(2), out_dtype=1, stream=None),
    "ma_mx4_matmul": dict(xq=at(0), xscale=at(1), x_bits=4, rows=100, wq=at(2), wscale=at(3), outs=64, ins=300, y=at(4), y_dtype=1,
                          accumulate=0, workspace=at(5), workspace_bytes=1 << 33, stream=None),
}
INV, UNS, WS = L.MA_ERR_INVALID_ARG, L.MA_ERR_UNSUPPORTED, L.MA_ERR_WORKSPACE


def call(name, **kw):
    args = dict(CALLS[name])
    assert not set(kw) - set(args), kw
    args.update(kw)
    return getattr(L.lib(), name)(*args.values())


F, B, P, U, M = "ma_rmsnorm_forward", "ma_rmsnorm_backward", "ma_mx4_pack", "ma_mx4_unpack", "ma_mx4_matmul"
BAD = [
    (F, dict(cols=16385), INV), (F, dict(cols=0), INV), (F, dict(rows=-1), INV), (F, dict(rows=(1 << 24) + 1), INV), (F, dict(rows=1 << 24, cols=4097), INV),
    (F, dict(eps=-1.0), INV), (F, dict(eps=float("nan")), INV), (F, dict(eps=float("inf")), INV), (F, dict(x=None), INV), (F, dict(rstd=None), INV),
    (F, dict(x_dtype=2), UNS), (F, dict(residual_dtype=5), UNS), (F, dict(y_dtype=7), UNS), (F, dict(total=None), INV), (F, dict(residual=None), INV),
    (F, dict(held_q=None), INV), (F, dict(held_scale=None), INV), (F, dict(y=None, held_q=None, held_scale=None), INV),
    (F, dict(held_q=at(6) + 8), INV), (F, dict(gain=at(2) + 2), INV), (F, dict(x=at(0) + 1), INV), (F, dict(total=at(3) + 2), INV),
    (F, dict(total=at(1)), INV), (F, dict(total=at(0)), INV), (F, dict(y=at(0)), INV), (F, dict(y=at(3) + 4), INV), (F, dict(rstd=at(2)), INV),
    (F, dict(held_q=at(4)), INV), (F, dict(rstd=at(5) + 2), INV),
    (B, dict(dy=None), INV), (B, dict(t=None), INV), (B, dict(t=None, held_q=at(8)), INV), (B, dict(held_q=at(8), held_scale=at(9)), INV),
    (B, dict(dx=None), INV), (B, dict(rstd=None), INV), (B, dict(dy_dtype=3), UNS), (B, dict(t_dtype=3), UNS), (B, dict(dx_dtype=0), UNS),
    (B, dict(t=None, held_q=at(8), held_scale=at(9), dy_dtype=0, dx_dtype=1), UNS), (B, dict(dx=at(0)), INV), (B, dict(dx=at(4)), INV),
    (B, dict(dx=at(1)), INV), (B, dict(dgain=at(3)), INV), (B, dict(dtotal=at(4) + 1), INV), (B, dict(accumulate=2), INV), (B, dict(cols=16385), INV),
    (B, dict(rows=1100, workspace=None), WS), (B, dict(rows=1100, workspace_bytes=8), WS), (B, dict(rows=1100, workspace=at(7) + 16), WS),
    (B, dict(rows=1100, workspace=at(5)), INV),
    (P, dict(x=None), INV), (P, dict(q=None), INV), (P, dict(scale=None), INV), (P, dict(q=at(1) + 8), INV), (P, dict(scale=at(2) + 2), INV),
    (P, dict(x_dtype=2), UNS), (P, dict(transpose=2), INV), (P, dict(transpose=-1), INV), (P, dict(cols=0), INV), (P, dict(rows=-1), INV),
    (P, dict(q=at(0)), INV), (P, dict(scale=at(1) + 64), INV), (P, dict(x=at(0) + 1), INV), (P, dict(rows=1 << 24, cols=4097), INV),
    (P, dict(rows=1 << 24, cols=(1 << 11) + 1, x_dtype=0), INV), (P, dict(rows=(1 << 11) + 1, cols=1 << 24, x_dtype=0, transpose=1), INV),
    (P, dict(rows=1, cols=1 << 24, transpose=1, x_dtype=0), None), (P, dict(rows=5, cols=(1 << 24) + 1), INV),
    (U, dict(q=None), INV), (U, dict(out=None), INV), (U, dict(out_dtype=3), UNS), (U, dict(out=at(0)), INV), (U, dict(out=at(2) + 1), INV),
    (U, dict(scale=at(1) + 1), INV), (U, dict(rows=1 << 24, cols=4097), INV),
    (M, dict(xq=None), INV), (M, dict(xscale=None), INV), (M, dict(wq=None), INV), (M, dict(wscale=None), INV), (M, dict(y=None), INV),
    (M, dict(x_bits=6), UNS), (M, dict(x_bits=0), UNS), (M, dict(y_dtype=2), UNS), (M, dict(accumulate=2), INV), (M, dict(rows=-1), INV),
    (M, dict(outs=0), INV), (M, dict(ins=0), INV), (M, dict(outs=(1 << 23) + 1), INV), (M, dict(ins=(1 << 23) + 1), INV), (M, dict(rows=(1 << 24) + 1), INV),
    (M, dict(rows=1 << 24, outs=4097), INV), (M, dict(rows=1 << 24, ins=4097), INV), (M, dict(outs=1 << 23, ins=8193), INV),
    (M, dict(xq=at(0) + 8), INV), (M, dict(wq=at(2) + 4), INV), (M, dict(wscale=at(3) + 1), INV), (M, dict(xscale=at(1) + 2), INV), (M, dict(y=at(4) + 1), INV),
    (M, dict(y=at(0)), INV), (M, dict(y=at(1)), INV), (M, dict(y=at(2) + 2), INV), (M, dict(y=at(3)), INV),
]


@pytest.mark.parametrize("name,kw,code", [b for b in BAD if b[2] is not None])
def test_rejects_bad_arguments(name, kw, code):
    assert call(name, **kw) == code
    assert L.lib().ma_last_error()


def test_empty_calls_are_no_ops():
    assert call(F, rows=0, x=None, residual=None, total=None, y=None, rstd=None, held_q=None, held_scale=None) == 0
    assert call(B, rows=0, dy=None, t=None, rstd=None, dx=None, dtotal=None, accumulate=1) == 0
    assert call(P, rows=0, x=None, q=None, scale=None) == 0
    assert call(U, rows=0, q=None, scale=None, out=None) == 0
    assert call(M, rows=0, xq=None, xscale=None, y=None) == 0


def test_workspace_sizes():
    assert ma.rmsnorm_workspace_size(0, 64) == 0 and ma.rmsnorm_workspace_size(1024, 64) == 0 and ma.rmsnorm_workspace_size(5000, 64) >= 64 * 4
    for f, a in ((ma.rmsnorm_workspace_size, (5, 1 << 20)), (ma.rmsnorm_workspace_size, (-1, 5)), (ma.rmsnorm_workspace_size, (1 << 24, 16384)),
                 (ma.mx4_matmul_workspace_size, (-1, 4, 4)), (ma.mx4_matmul_workspace_size, (4, 0, 4)), (ma.mx4_matmul_workspace_size, (4, 4, 0)),
                 (ma.mx4_matmul_workspace_size, (4, 4, 4, 5)), (ma.mx4_matmul_workspace_size, (1 << 24, 1 << 13, 4)),
                 (ma.mx4_matmul_workspace_size, (4, 1 << 23, 1 << 14))):
        with pytest.raises(ma.MuonAdamWError):
            f(*a)
    assert ma.mx4_matmul_workspace_size(0, 4, 4) == 0
    for cols in (1, 700, 1500, 2047, 4096, 8192, 16384):
        sizes = [ma.rmsnorm_workspace_size(rows, cols) for rows in [*range(0, 3000, 7), 4096, 5000, 20000, 49152, 1 << 20]]
        assert sizes == sorted(sizes)


def plan(rows, outs, ins, bits):
    e, s = C.c_int32(-1), C.c_int32(-1)
    assert L.lib().ma_test_mx4_matmul_plan(rows, outs, ins, bits, C.byref(e), C.byref(s)) == 0
    return e.value, s.value


def test_product_plan_query():
    """The query says what the workspace sizes say, and rejects what they reject."""
    for sizes in ((0, 4, 4), (1, 1, 1), (1, 16384, 4096), (129, 1003, 333), (12288, 16384, 4096), (900, 521, 20000), (2000, 2050, 9000), (1 << 24, 1, 1 << 12),
                  (1, 1 << 23, 1 << 13), (1 << 24, 4096, 1)):
        for bits in (4, 8):
            edge, splits = plan(*sizes, bits)
            assert edge in (0, 128, 256) and 1 <= splits <= -(-sizes[2] // 128) and (edge or splits == 1)
            assert ma.mx4_matmul_workspace_size(*sizes, bits) == (0 if splits == 1 else splits * -(-sizes[0] * sizes[1] // 64) * 64 * 4)
    assert plan(1, 16384, 4096, 8) == (0, 1) and plan(12288, 16384, 4096, 4) == (256, 1) and plan(900, 521, 20000, 4)[1] > 1
    e, f = C.c_int32(), L.lib().ma_test_mx4_matmul_plan
    assert f(-1, 4, 4, 4, C.byref(e), C.byref(e)) == INV and f(4, 0, 4, 4, C.byref(e), C.byref(e)) == INV and f(4, 4, 4, 5, C.byref(e), C.byref(e)) == UNS
    assert f(4, 4, 4, 4, None, C.byref(e)) == INV and f(4, 4, 4, 4, C.byref(e), None) == INV


def test_a_product_that_needs_a_workspace_rejects_a_small_one():
    need = ma.mx4_matmul_workspace_size(900, 521, 20000)
    assert need > 0
    for kw in (dict(workspace=None), dict(workspace_bytes=need - 1), dict(workspace=at(5) + 64)):
        assert call(M, rows=900, outs=521, ins=20000, **kw) == WS
    assert call(M, rows=900, outs=521, ins=20000, workspace=at(4) + 256) == INV
    assert call(M, rows=900, outs=521, ins=20000, workspace=at(2)) == INV


def test_binding_rejects_wrong_tensors():
    f32, bf, u8 = torch.float32, torch.bfloat16, torch.uint8
    x, c, st = torch.zeros(4, 8), ma.ActCheckpoint.empty(4, 8, "cpu"), torch.zeros(4)
    m, w = ma.Mx4Matrix.empty(4, 8, "cpu"), ma.Mx4Matrix.empty(6, 8, "cpu")
    T, V = TypeError, ValueError
    for err, f, a, kw in [
        (T, ma.rmsnorm_forward, (x.half(),), {}), (T, ma.rmsnorm_forward, (x, torch.zeros(8, dtype=bf)), {}), (V, ma.rmsnorm_forward, (x, torch.zeros(7)), {}),
        (V, ma.rmsnorm_forward, (x, None, x[:3]), {}), (T, ma.rmsnorm_forward, (x, None, x.half()), {}), (V, ma.rmsnorm_forward, (x,), dict(total=x)),
        (T, ma.rmsnorm_forward, (x, None, x), dict(total=x.bfloat16())), (V, ma.rmsnorm_forward, (x, None, x), dict(total=x[:2])),
        (V, ma.rmsnorm_forward, (x,), dict(rstd=torch.zeros(4, 2))), (T, ma.rmsnorm_forward, (x,), dict(rstd=st.double())),
        (T, ma.rmsnorm_forward, (x,), dict(held=x)), (V, ma.rmsnorm_forward, (x,), dict(held=ma.ActCheckpoint.empty(5, 8, "cpu"))),
        (V, ma.rmsnorm_forward, (x,), dict(held=c, dtype=bf)), (T, ma.rmsnorm_forward, (x,), dict(dtype=torch.float16)),
        (T, ma.rmsnorm_forward, (x,), dict(out=x.bfloat16(), dtype=f32)), (V, ma.rmsnorm_forward, (torch.zeros(8, 8)[:, ::2],), {}),
        (V, ma.rmsnorm_forward, (torch.zeros(4, 0),), {}), (T, ma.rmsnorm_forward, ([1.0],), {}),
        (V, ma.rmsnorm_backward, (x, x[:2], st), {}), (V, ma.rmsnorm_backward, (x, x, st[:3]), {}), (T, ma.rmsnorm_backward, (x, x, st), dict(dx=x.bfloat16())),
        (T, ma.rmsnorm_backward, (x, x, st), dict(dtotal=x.bfloat16())), (V, ma.rmsnorm_backward, (x, c, st), dict(dgain=torch.zeros(9))),
        (T, ma.rmsnorm_backward, (x.bfloat16(), c, st), dict(dx=x)), (T, ma.rmsnorm_backward, (x.bfloat16(), c, st), dict(dtotal=x)),
        (T, ma.rmsnorm_backward, (x, x, st), dict(dgain=torch.zeros(8), workspace=torch.zeros(9))), (V, ma.rmsnorm_backward, (x, ma.ActCheckpoint.empty(4, 9, "cpu"), st), {}),
        (T, ma.mx4_pack, (x.half(),), {}), (T, ma.mx4_pack, (x,), dict(out=c)), (V, ma.mx4_pack, (x,), dict(out=w)), (V, ma.mx4_pack, (x,), dict(out=m, transpose=True)),
        (V, ma.mx4_pack, (x.t(),), {}), (V, ma.mx4_pack, (x[:0],), dict(transpose=True)), (T, ma.mx4_unpack, (c,), {}), (T, ma.mx4_unpack, (m,), dict(dtype=torch.float16)),
        (V, ma.mx4_unpack, (m,), dict(out=torch.zeros(4, 9))),
        (T, ma.mx4_matmul, (x, w), {}), (T, ma.mx4_matmul, (m, c), {}), (V, ma.mx4_matmul, (ma.Mx4Matrix.empty(4, 9, "cpu"), w), {}),
        (V, ma.mx4_matmul, (m, w), dict(accumulate=True)), (V, ma.mx4_matmul, (m, w), dict(out=torch.zeros(4, 5))), (T, ma.mx4_matmul, (m, w), dict(dtype=torch.float16)),
        (T, ma.mx4_matmul, (m, w), dict(out=torch.zeros(4, 6), dtype=bf)), (V, ma.mx4_matmul, (c, w), dict(out=torch.zeros(6, 4).t())),
        (T, ma.mx4_matmul, (m, w), dict(workspace=torch.zeros(4))),
        (V, ma.Mx4Matrix, (torch.zeros(4, 64, dtype=u8), torch.zeros(4, 1, 4, dtype=u8), 8), {}), (V, ma.Mx4Matrix, (torch.zeros(4, 4, dtype=u8), m.scale, 8), {}),
        (T, ma.Mx4Matrix, (torch.zeros(4, 64), m.scale, 8), {}), (V, ma.Mx4Matrix, (m.q, m.scale, 0), {}), (V, ma.Mx4Matrix.empty, (4, 0, "cpu"), {}),
        (V, ma.Mx4Matrix.empty, (-1, 4, "cpu"), {}),
    ]:
        with pytest.raises(err):
            f(*a, **kw)


def test_binding_rejects_host_tensors():
    x, c, st = torch.zeros(4, 8), ma.ActCheckpoint.empty(4, 8, "cpu"), torch.zeros(4)
    m = ma.Mx4Matrix.empty(4, 8, "cpu")
    for f in (lambda: ma.rmsnorm_forward(x), lambda: ma.rmsnorm_forward(x, held=c), lambda: ma.rmsnorm_backward(x, x, st), lambda: ma.mx4_pack(x),
              lambda: ma.mx4_unpack(m), lambda: ma.mx4_matmul(m, m), lambda: ma.mx4_matmul(c, m)):
        with pytest.raises(ValueError, match="CUDA"):
            f()


def test_a_4_bit_matrix_is_two_tensors_or_one():
    m = ma.Mx4Matrix.empty(5, 130, "cpu")
    assert m.q.shape == (5, 128) and m.scale.shape == (2, 5, 4) and m.nbytes() == 5 * 128 + 40
    assert m._pointers() == (m.q.data_ptr(), m.scale.data_ptr())
    two = ma.Mx4Matrix(m.q, m.scale.clone(), 130)
    assert two._pointers() == (m.q.data_ptr(), two.scale.data_ptr()) and (two.rows, two.cols) == (5, 130)
