"""The fp64 oracle of the operators around the step, against independent
routines: torch's own float8 casts, embedding and layer norm on the CPU in
fp64, and central differences for the gradients."""
import numpy as np
import pytest
import torch

from oracle import train_ops as T


def test_e4m3_values_and_rounding_match_torch():
    q = np.arange(256, dtype=np.uint8)
    want = torch.from_numpy(q).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(T.e4m3_value(q), want, equal_nan=True)
    v = np.concatenate([np.linspace(-448, 448, 20001), 2.0 ** np.linspace(-12, 8, 5001),
                        (T._POSITIVE[1:] + T._POSITIVE[:-1]) / 2, T._POSITIVE, -T._POSITIVE, [-0.0]])
    got = T.e4m3_byte(v)
    v32 = v.astype(np.float32)   # torch rounds from fp32
    assert np.array_equal(T.e4m3_byte(v32), torch.from_numpy(v32).to(torch.float8_e4m3fn).view(torch.uint8).numpy())
    err = np.abs(T.e4m3_value(got) - v)
    assert np.all(err <= np.maximum(np.abs(v) * 2.0 ** -4, 2.0 ** -10))
    mids = (T._POSITIVE[1:] + T._POSITIVE[:-1]) / 2
    assert np.all(T.e4m3_byte(mids) % 2 == 0)


def test_checkpoint_exponent_is_the_least_that_holds_the_block():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((40, 128)) * 2.0 ** rng.integers(-100, 100, (40, 1))
    x[0] = 0
    x[1, :] = 0
    x[1, 5] = 448.0
    x[2, :] = 0
    x[2, 5] = np.nextafter(np.float32(448), np.float32(449))
    x[3, 7] = np.inf
    x[4, 9] = np.nan
    q, s = T.act_pack(x)
    e = s[:, 0].astype(int) - 127
    assert e[0] == T.ACT_EMIN and e[1] == 0 and e[2] == 1
    amax = np.abs(np.where(np.isfinite(x), x, 0)).max(1)
    assert np.all(amax <= 448 * 2.0 ** e) and np.all(amax[1:] > 448 * 2.0 ** (e[1:] - 1))
    back = T.act_unpack(q, s, 128)
    assert np.isnan(back[3, 7]) and np.isnan(back[4, 9]) and np.isnan(back).sum() == 2
    ok = np.isfinite(x)
    step = np.broadcast_to(2.0 ** e[:, None] * 2.0 ** -10, x.shape)
    assert np.all(np.abs(back - x)[ok] <= np.maximum(np.abs(x) * 2.0 ** -4, step)[ok])


def test_checkpoint_of_ragged_columns_and_the_largest_values():
    x = np.full((2, 130), 3.0)
    x[1, 129] = np.float64(np.finfo(np.float32).max)
    q, s = T.act_pack(x)
    assert q.shape == (2, 256) and s.shape == (2, 2) and not q[:, 130:].any()
    back = T.act_unpack(q, s, 130)
    assert np.all(np.isfinite(back.astype(np.float32))) and back[1, 129] == 240 * 2.0 ** 120
    assert np.array_equal(back[0], x[0]) and np.array_equal(back[1, :128], x[1, :128]) and back[1, 128] == 0


def test_every_held_value_is_exact_in_bf16():
    q = np.tile(np.arange(128, dtype=np.uint8)[:127], (238, 1))
    q = np.pad(q, ((0, 0), (0, 1)))
    s = np.arange(10, 248, dtype=np.uint8)[:, None]
    v = T.act_unpack(q, s, 128)
    v = v[:, :][np.abs(v) < 2.0 ** 128]     # beyond 240 * 2^120 nothing is packed
    assert np.array_equal(torch.from_numpy(v).to(torch.bfloat16).double().numpy(), v)


def test_embedding_matches_torch():
    g = torch.Generator().manual_seed(0)
    w = torch.randn(11, 7, generator=g, dtype=torch.float64, requires_grad=True)
    t = torch.randint(0, 11, (4, 5), generator=g)
    d = torch.randn(4, 5, 7, generator=g, dtype=torch.float64)
    y = torch.nn.functional.embedding(t, w) * 0.5
    y.backward(d)
    assert np.allclose(T.embedding_forward(w.detach().numpy(), t.numpy(), 0.5), y.detach().numpy(), rtol=1e-15)
    out, mag, count = T.embedding_backward(d.numpy(), t.numpy(), 11, 0.5)
    assert np.allclose(out, w.grad.numpy(), rtol=1e-13) and count.sum() == 20 and np.all(mag >= np.abs(out) - 1e-12)
    out2, _, c2 = T.embedding_backward(d.numpy(), np.where(t.numpy() > 5, -1, t.numpy()), 11, 0.5, grad=np.ones((11, 7)))
    assert np.all(out2[6:] == 1) and c2[6:].sum() == 0


@pytest.mark.parametrize("affine", [False, True])
def test_layernorm_gradients_match_central_differences(affine):
    rng = np.random.default_rng(1)
    x, dy = rng.standard_normal((3, 9)), rng.standard_normal((3, 9))
    gain, bias = (rng.standard_normal(9), rng.standard_normal(9)) if affine else (None, None)
    y, mean, rstd = T.layernorm_forward(x, gain, bias)
    ref = torch.nn.functional.layer_norm(torch.from_numpy(x), (9,), None if gain is None else torch.from_numpy(gain),
                                         None if bias is None else torch.from_numpy(bias), float(np.float32(1e-5))).numpy()
    assert np.allclose(y, ref, rtol=1e-12, atol=1e-13)
    dx, dgain, dbias = T.layernorm_backward(dy, x, mean, rstd, gain)
    loss = lambda x, gain, bias: (T.layernorm_forward(x, gain, bias)[0] * dy).sum()  # noqa: E731
    h = 1e-6

    def diff(f, v):
        out = np.zeros_like(v)
        for i in np.ndindex(*v.shape):
            p, m = v.copy(), v.copy()
            p[i] += h
            m[i] -= h
            out[i] = (f(p) - f(m)) / (2 * h)
        return out
    # central differences: h^2 |f'''| / 6 + 1e-16 |f| / h, both below 1e-8 here
    assert np.allclose(dx, diff(lambda v: loss(v, gain, bias), x), atol=1e-7)
    if affine:
        assert np.allclose(dgain, diff(lambda v: loss(x, v, bias), gain), atol=1e-7)
        assert np.allclose(dbias, diff(lambda v: loss(x, gain, v), bias), atol=1e-7)


def test_weight_grad_matches_torch():
    rng = np.random.default_rng(2)
    x, dy, w = rng.standard_normal((6, 5)), rng.standard_normal((6, 4)), torch.zeros(4, 5, dtype=torch.float64, requires_grad=True)
    (torch.from_numpy(x) @ w.t() * torch.from_numpy(dy)).sum().backward()
    out, mag = T.act_weight_grad(dy, x)
    assert np.allclose(out, w.grad.numpy(), rtol=1e-13) and np.all(mag >= np.abs(out))
    assert np.allclose(T.act_weight_grad(dy, x, np.ones((4, 5)))[0], out + 1)
