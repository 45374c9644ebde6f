"""The operators around the step without a GPU: every entry point rejects bad
arguments before any launch (these calls never reach the HIP runtime), and the
binding rejects wrong types, shapes, strides and host tensors."""
import ctypes as C
import os

import pytest
import torch

import adamw_optimizer_step_amd as ma
from adamw_optimizer_step_amd import _lib as L

pytestmark = pytest.mark.skipif(not os.path.exists(L.LIB_PATH), reason="library not built")

BASE, GAP = 1 << 40, 1 << 34   # fake, never dereferenced device addresses
at = lambda i: BASE + i * GAP  # noqa: E731

CALLS = {
    "ma_embedding_forward": dict(table=at(0), table_dtype=0, rows=100, cols=64, tokens=at(1), token_bytes=8, n_tokens=10, scale=1.0,
                                 out=at(2), out_dtype=1, stream=None),
    "ma_embedding_backward": dict(dout=at(0), dout_dtype=1, tokens=at(1), token_bytes=8, n_tokens=10, rows=100, cols=64, scale=1.0,
                                  accumulate=0, grad=at(2), workspace=at(3), workspace_bytes=1 << 30, stream=None),
    "ma_layernorm_forward": dict(x=at(0), x_dtype=1, rows=10, cols=64, gain=at(1), bias=at(2), eps=1e-5, y=at(3), y_dtype=1,
                                 stats=at(4), ckpt_q=at(5), ckpt_scale=at(6), stream=None),
    "ma_layernorm_backward": dict(dy=at(0), dy_dtype=1, x=at(1), x_dtype=1, ckpt_q=None, ckpt_scale=None, rows=10, cols=64,
                                  stats=at(2), gain=at(3), dx=at(4), dx_dtype=1, dgain=at(5), dbias=at(6), accumulate=0,
                                  workspace=at(7), workspace_bytes=1 << 30, stream=None),
    "ma_act_pack": dict(x=at(0), x_dtype=1, rows=10, cols=64, q=at(1), scale=at(2), stream=None),
    "ma_act_unpack": dict(q=at(0), scale=at(1), rows=10, cols=64, out=at(2), out_dtype=1, stream=None),
    "ma_act_weight_grad": dict(dy=at(0), dy_dtype=1, q=at(1), scale=at(2), tokens=4096, outs=64, ins=64, grad=at(3), grad_dtype=1,
                               accumulate=0, workspace=at(4), workspace_bytes=1 << 33, stream=None),
}
INV, UNS, WS = L.MA_ERR_INVALID_ARG, L.MA_ERR_UNSUPPORTED, L.MA_ERR_WORKSPACE


def call(name, **kw):
    args = dict(CALLS[name])
    assert not set(kw) - set(args), kw
    args.update(kw)
    return getattr(L.lib(), name)(*args.values())


BAD = [
    ("ma_embedding_forward", dict(rows=0), INV), ("ma_embedding_forward", dict(cols=0), INV),
    ("ma_embedding_forward", dict(rows=(1 << 24) + 1), INV), ("ma_embedding_forward", dict(cols=(1 << 24) + 1), INV),
    ("ma_embedding_forward", dict(rows=1 << 24, cols=1 << 15), INV), ("ma_embedding_forward", dict(rows=1 << 24, cols=2049), INV), ("ma_embedding_forward", dict(n_tokens=-1), INV),
    ("ma_embedding_forward", dict(n_tokens=(1 << 25) + 1), INV), ("ma_embedding_forward", dict(table_dtype=2), UNS),
    ("ma_embedding_forward", dict(out_dtype=-1), UNS), ("ma_embedding_forward", dict(token_bytes=2), UNS),
    ("ma_embedding_forward", dict(scale=float("nan")), INV), ("ma_embedding_forward", dict(table=None), INV),
    ("ma_embedding_forward", dict(tokens=None), INV), ("ma_embedding_forward", dict(out=None), INV),
    ("ma_embedding_forward", dict(table=at(0) + 2), INV), ("ma_embedding_forward", dict(out=at(2) + 1), INV),
    ("ma_embedding_forward", dict(tokens=at(1) + 4), INV), ("ma_embedding_forward", dict(out=at(0)), INV),
    ("ma_embedding_backward", dict(dout=None), INV), ("ma_embedding_backward", dict(grad=None), INV),
    ("ma_embedding_backward", dict(accumulate=2), INV), ("ma_embedding_backward", dict(scale=float("inf")), INV),
    ("ma_embedding_backward", dict(token_bytes=1), UNS), ("ma_embedding_backward", dict(dout_dtype=3), UNS),
    ("ma_embedding_backward", dict(workspace=None), WS), ("ma_embedding_backward", dict(workspace_bytes=100), WS),
    ("ma_embedding_backward", dict(workspace=at(3) + 8), WS), ("ma_embedding_backward", dict(grad=at(0)), INV),
    ("ma_embedding_backward", dict(workspace=at(2)), INV), ("ma_embedding_backward", dict(grad=at(1) + 64), INV),
    ("ma_layernorm_forward", dict(cols=16385), INV), ("ma_layernorm_forward", dict(rows=-1), INV),
    ("ma_layernorm_forward", dict(eps=-1.0), INV), ("ma_layernorm_forward", dict(eps=float("nan")), INV),
    ("ma_layernorm_forward", dict(x=None), INV), ("ma_layernorm_forward", dict(stats=None), INV),
    ("ma_layernorm_forward", dict(stats=at(4) + 4), INV), ("ma_layernorm_forward", dict(gain=at(1) + 2), INV),
    ("ma_layernorm_forward", dict(ckpt_q=None), INV), ("ma_layernorm_forward", dict(ckpt_scale=None), INV),
    ("ma_layernorm_forward", dict(ckpt_q=at(5) + 8), INV), ("ma_layernorm_forward", dict(y=at(0)), INV),
    ("ma_layernorm_forward", dict(y=at(1)), INV), ("ma_layernorm_forward", dict(ckpt_q=at(0)), INV),
    ("ma_layernorm_forward", dict(y_dtype=7), UNS),
    ("ma_layernorm_backward", dict(dx_dtype=0), UNS), ("ma_layernorm_backward", dict(dy_dtype=5), UNS),
    ("ma_layernorm_backward", dict(x=None), INV), ("ma_layernorm_backward", dict(x=None, ckpt_q=at(8)), INV),
    ("ma_layernorm_backward", dict(ckpt_q=at(8), ckpt_scale=at(9)), INV), ("ma_layernorm_backward", dict(stats=None), INV),
    ("ma_layernorm_backward", dict(dx=at(0)), INV), ("ma_layernorm_backward", dict(dgain=at(6)), INV),
    ("ma_layernorm_backward", dict(rows=1100, workspace=None), WS), ("ma_layernorm_backward", dict(rows=1100, workspace_bytes=8), WS),
    ("ma_layernorm_backward", dict(accumulate=-1), INV),
    ("ma_layernorm_backward", dict(x=None, ckpt_q=at(8), ckpt_scale=at(9), dy_dtype=0, dx_dtype=1), UNS),
    ("ma_act_pack", dict(x=None), INV), ("ma_act_pack", dict(q=at(1) + 4), INV), ("ma_act_pack", dict(q=at(0)), INV),
    ("ma_act_pack", dict(x_dtype=2), UNS), ("ma_act_pack", dict(cols=0), INV), ("ma_act_pack", dict(scale=None), INV),
    ("ma_act_pack", dict(rows=1 << 24, cols=(1 << 14) + 1), INV), ("ma_act_pack", dict(rows=1 << 24, cols=(1 << 11) + 1, x_dtype=0), INV),
    ("ma_act_unpack", dict(out=at(0)), INV), ("ma_act_unpack", dict(out_dtype=4), UNS), ("ma_act_unpack", dict(out=at(2) + 1), INV),
    ("ma_act_unpack", dict(q=None), INV),
    ("ma_act_weight_grad", dict(dy=None), INV), ("ma_act_weight_grad", dict(q=None), INV), ("ma_act_weight_grad", dict(scale=None), INV),
    ("ma_act_weight_grad", dict(grad=None), INV), ("ma_act_weight_grad", dict(grad=at(0)), INV), ("ma_act_weight_grad", dict(grad=at(1)), INV),
    ("ma_act_weight_grad", dict(outs=0), INV), ("ma_act_weight_grad", dict(ins=-1), INV), ("ma_act_weight_grad", dict(tokens=-1), INV),
    ("ma_act_weight_grad", dict(outs=1 << 16, ins=(1 << 15) + 1), INV), ("ma_act_weight_grad", dict(grad_dtype=2), UNS),
    ("ma_act_weight_grad", dict(dy_dtype=2), UNS), ("ma_act_weight_grad", dict(accumulate=3), INV),
    ("ma_act_weight_grad", dict(q=at(1) + 1), INV),
]


@pytest.mark.parametrize("name,kw,code", [b for b in BAD if b[2] is not None])
def test_rejects_bad_arguments(name, kw, code):
    assert call(name, **kw) == code
    assert L.lib().ma_last_error()


def test_empty_calls_are_no_ops():
    assert call("ma_embedding_forward", n_tokens=0, tokens=None, out=None) == 0
    assert call("ma_embedding_backward", n_tokens=0, dout=None, tokens=None, accumulate=1) == 0
    assert call("ma_layernorm_forward", rows=0, x=None, y=None, stats=None, ckpt_q=None, ckpt_scale=None) == 0
    assert call("ma_layernorm_backward", rows=0, x=None, dy=None, dx=None, stats=None, accumulate=1) == 0
    assert call("ma_act_pack", rows=0, x=None, q=None, scale=None) == 0
    assert call("ma_act_unpack", rows=0, out=None, q=None, scale=None) == 0
    assert call("ma_act_weight_grad", tokens=0, dy=None, q=None, scale=None, accumulate=1) == 0


def test_workspace_sizes():
    assert ma.embedding_workspace_size(100, 64, 0) >= 256
    assert ma.embedding_workspace_size(50304, 1024, 49152) >= 2 * 4 * (50304 + 49152)
    assert ma.layernorm_workspace_size(0, 64) == 0 and ma.layernorm_workspace_size(1, 64) == 0 and ma.layernorm_workspace_size(5000, 64) >= 2 * 64 * 4
    assert ma.act_weight_grad_workspace_size(0, 4, 4) == 0
    for f, a in ((ma.embedding_workspace_size, (0, 1, 1)), (ma.layernorm_workspace_size, (5, 1 << 20)),
                 (ma.act_weight_grad_workspace_size, (5, 0, 3)), (ma.layernorm_workspace_size, (1 << 24, 16384)),
                 (ma.act_weight_grad_workspace_size, (1 << 26, 4, 4)), (ma.act_weight_grad_workspace_size, (5, 1 << 24, 4)),
                 (ma.act_weight_grad_workspace_size, (5, 1 << 20, 1 << 20)), (ma.act_weight_grad_workspace_size, (1 << 20, 4, 1 << 20))):
        with pytest.raises(ma.MuonAdamWError):
            f(*a)


def test_binding_rejects_wrong_tensors():
    f32, bf, i64 = torch.float32, torch.bfloat16, torch.int64
    W, t, d, x = torch.zeros(10, 8), torch.zeros(4, dtype=i64), torch.zeros(4, 8), torch.zeros(4, 8)
    c = ma.ActCheckpoint.empty(4, 8, "cpu")
    st = torch.zeros(4, 2)
    T, V = TypeError, ValueError
    for err, f, a, kw in [
        (T, ma.embedding_forward, (W.half(), t), {}), (T, ma.embedding_forward, (W, t.float()), {}),
        (T, ma.embedding_forward, (W, t), dict(dtype=torch.float16)), (V, ma.embedding_forward, (W[0], t), {}),
        (V, ma.embedding_forward, (W.t(), t), {}), (V, ma.embedding_forward, (W, t), dict(out=torch.zeros(3, 8))),
        (T, ma.embedding_forward, (W, t), dict(out=torch.zeros(4, 8), dtype=bf)), (V, ma.embedding_forward, (W, torch.zeros(8, dtype=i64)[::2]), {}),
        (T, ma.embedding_backward, (d, t, W.bfloat16()), {}), (V, ma.embedding_backward, (d[:3], t, W), {}),
        (V, ma.embedding_backward, (d, t, torch.zeros(10, 9)), {}), (T, ma.embedding_backward, (d, t, W), dict(workspace=torch.zeros(9))),
        (T, ma.layernorm_forward, (x.double(),), {}), (T, ma.layernorm_forward, (x, torch.zeros(8, dtype=bf)), {}),
        (V, ma.layernorm_forward, (x, torch.zeros(7)), {}), (V, ma.layernorm_forward, (x, None, None), dict(stats=torch.zeros(2, 4))),
        (V, ma.layernorm_forward, (x,), dict(checkpoint=ma.ActCheckpoint.empty(5, 8, "cpu"))), (T, ma.layernorm_forward, (x,), dict(checkpoint=x)),
        (V, ma.layernorm_forward, (torch.zeros(4, 0),), {}), (V, ma.layernorm_forward, (torch.zeros(8, 8)[:, ::2],), {}),
        (V, ma.layernorm_backward, (x, x[:2], st), {}), (V, ma.layernorm_backward, (x, x, st[:3]), {}),
        (T, ma.layernorm_backward, (x, x, st), dict(dx=x.bfloat16())), (V, ma.layernorm_backward, (x, c, st), dict(dgain=torch.zeros(9))),
        (T, ma.layernorm_backward, (x.bfloat16(), c, st), dict(dx=x)),
        (T, ma.act_pack, (x.half(),), {}), (V, ma.act_pack, (x,), dict(out=ma.ActCheckpoint.empty(4, 9, "cpu"))), (T, ma.act_unpack, (x,), {}),
        (T, ma.act_unpack, (c,), dict(dtype=torch.float16)), (V, ma.act_unpack, (c,), dict(out=torch.zeros(4, 9))),
        (V, ma.act_weight_grad, (torch.zeros(5, 6), c, torch.zeros(6, 8)), {}), (V, ma.act_weight_grad, (torch.zeros(4, 6), c, torch.zeros(8, 6)), {}),
        (T, ma.act_weight_grad, (torch.zeros(4, 6), x, torch.zeros(6, 8)), {}),
        (V, ma.ActCheckpoint, (torch.zeros(4, 8, dtype=torch.uint8), c.scale, 8), {}), (V, ma.ActCheckpoint, (c.q, c.scale, 0), {}),
        (T, ma.ActCheckpoint, (c.q.int(), c.scale, 8), {}),
    ]:
        with pytest.raises(err):
            f(*a, **kw)


def test_binding_rejects_host_tensors():
    W, t, x = torch.zeros(10, 8), torch.zeros(4, dtype=torch.int32), torch.zeros(4, 8)
    c, st = ma.ActCheckpoint.empty(4, 8, "cpu"), torch.zeros(4, 2)
    for f in (lambda: ma.embedding_forward(W, t), lambda: ma.embedding_backward(x, t, W), lambda: ma.layernorm_forward(x),
              lambda: ma.layernorm_backward(x, x, st), lambda: ma.act_pack(x), lambda: ma.act_unpack(c),
              lambda: ma.act_weight_grad(torch.zeros(4, 6), c, torch.zeros(6, 8))):
        with pytest.raises(ValueError, match="CUDA"):
            f()


def plan(t, n, k, dt):
    e, s = C.c_int32(-1), C.c_int32(-1)
    assert L.lib().ma_test_act_weight_grad_plan(t, n, k, dt, C.byref(e), C.byref(s)) == 0
    return e.value, s.value


def test_weight_grad_plan_query():
    """The query says what the workspace sizes say, and rejects what they reject."""
    for t, n, k in ((0, 4, 4), (1, 1, 1), (1000, 250, 333), (4099, 2050, 2041), (12288, 16384, 4096), (700, 4090, 4081), (63, 130, 300)):
        for dt, name in ((L.MA_F32, torch.float32), (L.MA_BF16, torch.bfloat16)):
            edge, splits = plan(t, n, k, dt)
            assert edge in (128, 256) and splits >= 1
            assert ma.act_weight_grad_workspace_size(t, n, k, name) == (0 if splits == 1 else splits * -(-n * k // 64) * 64 * 4)
    assert plan(12288, 16384, 4096, L.MA_BF16) == (256, 1) and plan(63, 130, 300, L.MA_BF16) == (128, 1)
    e = C.c_int32()
    f = L.lib().ma_test_act_weight_grad_plan
    assert f(-1, 4, 4, 0, C.byref(e), C.byref(e)) == INV and f(4, 0, 4, 0, C.byref(e), C.byref(e)) == INV
    assert f(4, 4, 4, 2, C.byref(e), C.byref(e)) == UNS and f(4, 4, 4, 0, None, C.byref(e)) == INV and f(4, 4, 4, 0, C.byref(e), None) == INV


def test_embedding_workspace_of_more_tokens_serves_fewer():
    """The size never falls with the tokens, past the changes of the pieces' length and of the form too."""
    for rows, cols in ((1, 1), (1000, 40), (50304, 1024), (1 << 18, 3)):
        sizes = [ma.embedding_workspace_size(rows, cols, n) for n in (0, 1, 1024, 1025, 3000, 16383, 16384, 16385, 20000, 30000, 32768, 32769, 49152, 1 << 20)]
        assert sizes == sorted(sizes)


def test_layernorm_workspace_of_more_rows_serves_fewer():
    for cols in (1, 700, 1500, 2047, 4096, 8192, 16384):
        sizes = [ma.layernorm_workspace_size(rows, cols) for rows in [*range(0, 3000, 7), 4096, 5000, 20000, 49152, 1 << 20]]
        assert sizes == sorted(sizes)


def test_a_workspace_that_is_too_small_is_named_as_such():
    """Also where the room it lacks belongs to another buffer of the call."""
    for name, kw in (("ma_embedding_backward", dict(n_tokens=5000, grad=at(3) + 256)),
                     ("ma_layernorm_backward", dict(rows=2000, workspace=at(3), dgain=at(3) + 256)),
                     ("ma_act_weight_grad", dict(workspace=at(4), grad=at(4) + 256))):
        assert call(name, workspace_bytes=256, **kw) == WS
        assert b"256 bytes" in L.lib().ma_last_error()
