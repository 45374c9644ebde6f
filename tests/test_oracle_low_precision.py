"""The fp64 oracle of root-mean-square norm and of 4-bit matrices against
independent routines: torch's norm and casts, the format's table of values and
central differences."""
import numpy as np
import pytest
import torch

from oracle import train_ops as T


def test_bf16_rounding_matches_torch():
    rng = np.random.default_rng(0)
    v = (rng.standard_normal(4000) * 2.0 ** rng.integers(-130, 120, 4000)).astype(np.float32)
    v[:4] = [np.inf, -np.inf, np.nan, 0.0]
    assert np.array_equal(T.bf16_nearest(v), torch.from_numpy(v).bfloat16().float().numpy(), equal_nan=True)


@pytest.mark.parametrize("gain,residual", [(False, False), (True, True), (True, False)])
def test_rmsnorm_matches_torch_and_central_differences(gain, residual):
    rng = np.random.default_rng(1)
    x, dy, dt = rng.standard_normal((3, 3, 9)).astype(np.float32).astype(np.float64)
    w = rng.standard_normal(9) if gain else None
    r = rng.standard_normal((3, 9)).astype(np.float32).astype(np.float64) if residual else None
    y, t, rstd = T.rmsnorm_forward(x, w, r)
    assert np.array_equal(t, x if r is None else (x.astype(np.float32) + r.astype(np.float32)).astype(np.float64))
    ref = torch.nn.functional.rms_norm(torch.from_numpy(t), (9,), None if w is None else torch.from_numpy(w), float(np.float32(1e-5)))
    assert np.allclose(y, ref.numpy(), rtol=1e-12, atol=1e-13)
    dx, dgain = T.rmsnorm_backward(dy, t, rstd, w, dt)
    loss = lambda t, w: (T.rmsnorm_forward(t, w)[0] * dy).sum() + (t * dt).sum()  # noqa: E731
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
    assert np.allclose(dx, diff(lambda v: loss(v, w), t), atol=1e-7)
    if gain:
        assert np.allclose(dgain, diff(lambda v: loss(t, v), w), atol=1e-7)


def test_a_bf16_stream_is_what_the_norm_reads():
    rng = np.random.default_rng(2)
    x, r = rng.standard_normal((2, 4, 32)).astype(np.float32)
    _, t, _ = T.rmsnorm_forward(x, None, r, bf16_stream=True)
    assert np.array_equal(t, torch.from_numpy(x + r).bfloat16().double().numpy())


def test_e2m1_values_ties_and_saturation():
    assert list(T.E2M1) == [0, 0.5, 1, 1.5, 2, 3, 4, 6]
    for c in range(8):     # sign, 2 bits of exponent with bias 1, 1 of fraction
        e, f = c >> 1, c & 1
        assert T.E2M1[c] == ((1 + f / 2) * 2.0 ** (e - 1) if e else f / 2)
    assert np.array_equal(T.e2m1_code(T.E2M1), np.arange(8)) and np.array_equal(T.e2m1_code(-T.E2M1), np.arange(8) + 8)
    mids = (T.E2M1[1:] + T.E2M1[:-1]) / 2
    assert list(T.e2m1_code(mids)) == [0, 2, 2, 4, 4, 6, 6]
    assert list(T.e2m1_code(np.nextafter(mids, 9))) == list(range(1, 8)) and list(T.e2m1_code(np.nextafter(mids, 0))) == list(range(7))
    assert list(T.e2m1_code([6.9, 8.0, -1e9])) == [7, 7, 15]


def test_mx4_exponent_is_the_least_that_holds_the_block():
    rng = np.random.default_rng(3)
    x = rng.standard_normal((60, 128)) * 2.0 ** rng.integers(-100, 100, (60, 1))
    x[0] = 0
    x[1, :32] = 0
    x[1, 5] = np.nextafter(np.float32(7), np.float32(0))
    x[2, :32] = 0
    x[2, 5] = 7.0
    x[3, 40], x[4, 127] = np.inf, np.nan
    q, s = T.mx4_pack(x)
    assert q.shape == (60, 64) and s.shape == (1, 60, 4)
    assert (s[0, 0] == 1).all() and s[0, 1, 0] == 127 and s[0, 2, 0] == 128
    assert s[0, 3, 1] == 255 and s[0, 4, 3] == 255 and (s == 255).sum() == 2
    back = T.mx4_unpack(q, s, 128)
    assert np.isnan(back[3, 32:64]).all() and np.isnan(back[4, 96:]).all() and np.isnan(back).sum() == 64
    step = np.where(s == 255, np.nan, 2.0 ** (s.astype(float) - 127))[0].repeat(32, 1)
    with np.errstate(invalid="ignore"):
        ok = np.isfinite(back)
        # in [2^k, 2^(k+1)) values are 2^(k-1) apart: off by 2^(k-2) at most, first at 1.25 * 2^k; from 6 to 7, by 1
        assert np.all((np.abs(back - x) <= np.maximum(np.abs(x) / 5, step / 4))[ok])
        amax = np.abs(np.where(ok, x, 0)).reshape(60, 4, 32).max(-1)
        e = step.reshape(60, 4, 32)[..., 0]
        assert np.all((amax < 7 * e)[np.isfinite(e)]) and np.all((amax >= 3.5 * e)[np.isfinite(e) & (amax > 0)])


def test_mx4_of_ragged_columns_and_the_largest_values():
    x = np.full((3, 130), 3.0)
    x[1, 129] = np.float64(np.finfo(np.float32).max)
    x[2, 129] = 2.0 ** -149
    q, s = T.mx4_pack(x)
    assert q.shape == (3, 128) and s.shape == (2, 3, 4) and not q[:, 65:].any()
    back = T.mx4_unpack(q, s, 130)
    assert back[1, 129] == 6 * 2.0 ** 125 and np.isfinite(back.astype(np.float32)).all() and back[1, 128] == 0
    assert np.array_equal(back[0], x[0]) and back[2, 129] == 0 and back[2, 128] == 3


def test_every_value_held_in_4_bits_is_exact_in_bf16():
    q = np.tile(np.arange(256, dtype=np.uint8)[:64], (252, 1))
    q[:, 32:] = np.arange(192, 224)
    s = np.repeat(np.arange(1, 253, dtype=np.uint8)[None, :, None], 4, 2)
    v = T.mx4_unpack(q, s, 128)
    assert np.array_equal(torch.from_numpy(v).to(torch.bfloat16).double().numpy(), v)


def test_product_matches_torch():
    rng = np.random.default_rng(4)
    x, w, y = rng.standard_normal((5, 7)), rng.standard_normal((3, 7)), rng.standard_normal((5, 3))
    out, mag = T.mx4_matmul(x, w, y)
    assert np.allclose(out, torch.nn.functional.linear(torch.from_numpy(x), torch.from_numpy(w)).numpy() + y, rtol=1e-13)
    assert np.all(mag >= np.abs(out - y) - 1e-12)
