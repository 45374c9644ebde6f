"""The operators around the optimizer step in fp64, from their formulas:
embedding, layer norm, 8-bit activation checkpoints, the weight gradient."""
import numpy as np

ACT_BLOCK = 128
ACT_EMIN, ACT_EMAX = -117, 120


def embedding_forward(table, tokens, scale):
    table, tokens = np.asarray(table, np.float64), np.asarray(tokens)
    out = np.zeros(tokens.shape + table.shape[1:])
    for i in np.ndindex(*tokens.shape):
        if 0 <= tokens[i] < table.shape[0]:
            out[i] = table[tokens[i]] * float(np.float32(scale))
    return out


def embedding_backward(dout, tokens, rows, scale, grad=None):
    """``grad`` (zeros by default) plus each row's sum. Also returns how many
    tokens each row has and the sum of the magnitudes, for error bounds."""
    dout, tokens = np.asarray(dout, np.float64), np.asarray(tokens).reshape(-1)
    cols = dout.shape[-1]
    dout = dout.reshape(-1, cols)
    out = np.zeros((rows, cols)) if grad is None else np.array(grad, np.float64)
    mag, count = np.zeros((rows, cols)), np.zeros(rows, np.int64)
    ok = (tokens >= 0) & (tokens < rows)
    np.add.at(out, tokens[ok], dout[ok] * float(np.float32(scale)))
    np.add.at(mag, tokens[ok], np.abs(dout[ok]) * abs(float(np.float32(scale))))
    np.add.at(count, tokens[ok], 1)
    return out, mag, count


def layernorm_forward(x, gain=None, bias=None, eps=1e-5):
    x = np.asarray(x, np.float64)
    mean = x.mean(-1, keepdims=True)
    rstd = 1.0 / np.sqrt(((x - mean) ** 2).mean(-1, keepdims=True) + float(np.float32(eps)))
    y = (x - mean) * rstd
    if gain is not None:
        y = y * np.asarray(gain, np.float64)
    if bias is not None:
        y = y + np.asarray(bias, np.float64)
    return y, mean, rstd


def layernorm_backward(dy, x, mean, rstd, gain=None):
    """dx, dgain, dbias for given statistics."""
    dy, x = np.asarray(dy, np.float64), np.asarray(x, np.float64)
    xh = (x - mean) * rstd
    g = dy if gain is None else dy * np.asarray(gain, np.float64)
    dx = rstd * (g - g.mean(-1, keepdims=True) - xh * (g * xh).mean(-1, keepdims=True))
    return dx, (dy * xh).sum(0), dy.sum(0)


def e4m3_value(q):
    """fp64 values of e4m3 (OCP) bytes."""
    q = np.asarray(q, np.int64)
    e, f = (q >> 3) & 15, q & 7
    v = np.where(e > 0, (8.0 + f) * 2.0 ** (e - 10.0), f * 2.0 ** -9)
    v = np.where((q & 127) == 127, np.nan, v)
    return np.where(q & 128, -v, v)


_POSITIVE = e4m3_value(np.arange(127))   # 0 .. 448, increasing; the byte is the index


def e4m3_byte(v):
    """The e4m3 byte nearest to each v, |v| <= 448, ties to the even byte; NaN to 127."""
    v = np.asarray(v, np.float64)
    a = np.abs(np.where(np.isnan(v), 0.0, v))
    hi = np.clip(np.searchsorted(_POSITIVE, a), 1, 126)
    below, above = a - _POSITIVE[hi - 1], _POSITIVE[hi] - a
    q = np.where((below < above) | ((below == above) & (hi % 2 == 1)), hi - 1, hi)
    return (np.where(np.isnan(v), 127, q) | np.where(np.signbit(v) & ~np.isnan(v), 128, 0)).astype(np.uint8)


def act_pack(x):
    """(q, scale) bytes of the checkpoint of x [rows, cols]."""
    x = np.asarray(x, np.float64)
    rows, cols = x.shape
    blocks = -(-cols // ACT_BLOCK)
    v = np.zeros((rows, blocks * ACT_BLOCK))
    v[:, :cols] = x
    v = v.reshape(rows, blocks, ACT_BLOCK)
    amax = np.abs(np.where(np.isfinite(v), v, 0.0)).max(-1)
    e = np.full(amax.shape, ACT_EMIN)
    for k in range(ACT_EMIN, ACT_EMAX):           # the least exponent that holds amax
        e = np.where((e == k) & (amax > 448.0 * 2.0 ** k), k + 1, e)
    most = np.where(e == ACT_EMAX, 240.0, 448.0)[..., None]
    with np.errstate(invalid="ignore"):
        t = np.where(np.isfinite(v), np.clip(v / 2.0 ** e[..., None], -most, most), np.nan)
    return e4m3_byte(t).reshape(rows, -1), (e + 127).astype(np.uint8)


def act_unpack(q, scale, cols):
    rows, blocks = scale.shape
    s = 2.0 ** (scale.astype(np.float64) - 127)
    return (e4m3_value(q).reshape(rows, blocks, ACT_BLOCK) * s[..., None]).reshape(rows, -1)[:, :cols]


def act_weight_grad(dy, x, grad=None):
    """dy^T x (+ grad), and the sum of the products' magnitudes."""
    dy, x = np.asarray(dy, np.float64), np.asarray(x, np.float64)
    out = dy.T @ x
    return (out if grad is None else out + np.asarray(grad, np.float64)), np.abs(dy).T @ np.abs(x)
