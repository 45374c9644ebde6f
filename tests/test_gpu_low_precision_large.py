"""Calls of root-mean-square norm, 4-bit packing and the product whose operands pass the caches: their loads and stores
are non-temporal, in kernels that smaller calls do not run."""
import numpy as np
import pytest
import torch

import adamw_optimizer_step_amd as ma
from gpu_util import need_gpu, say, to_np
from oracle import train_ops as T
from test_gpu_low_precision import plan, rms_y_tol
from test_gpu_ops import BF16, DEV, F32, close, f64

pytestmark = pytest.mark.gpu
MIB = 1 << 20


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


def randn(shape, seed, dtype=F32):
    return torch.randn(shape, generator=torch.Generator(device=DEV).manual_seed(seed), device=DEV, dtype=F32).to(dtype)


@pytest.mark.parametrize("rows,outs,ins,edge", [(12289, 8201, 700, 256), (20001, 5203, 100, 128), (12289, 8201, 60, 128)])
@pytest.mark.parametrize("bits", [4, 8])
def test_product_with_a_bf16_result_past_the_caches(rows, outs, ins, edge, bits):
    """Sums of products of small whole numbers, exact in fp32, rounded once."""
    say("mx4_matmul, large bf16", rows, outs, ins, bits)
    assert rows * outs * 2 > 192 * MIB and plan(rows, outs, ins, bits) == (edge, 1)
    g = torch.Generator(device=DEV).manual_seed(300)
    table = torch.tensor([0, 1, 2, 3, 4, 6, -1, -2, -3, -4, -6], dtype=F32, device=DEV)
    xv, wv = (table[torch.randint(0, 11, (n, ins), generator=g, device=DEV)] for n in (rows, outs))
    xv[:, ::32], wv[:, ::32] = 6, -6      # every block's exponent 0
    x = ma.mx4_pack(xv) if bits == 4 else ma.act_pack(xv)
    want = torch.mm(xv.double(), wv.double().t()).float().bfloat16()
    assert torch.equal(ma.mx4_matmul(x, ma.mx4_pack(wv)), want)


@pytest.mark.parametrize("rows,cols", [(16400, 6200), (400001, 257), (65000, 1639)])
def test_packing_bf16_past_the_caches(rows, cols):
    say("mx4 bf16, large", rows, cols)
    assert rows * cols * 2 > 192 * MIB
    x = randn((rows, cols), 310, BF16)
    x[rows // 2, cols // 2], x[rows - 1] = float("nan"), 0
    m = ma.mx4_pack(x)
    out = ma.mx4_unpack(m)
    for a, b in ((0, 70), (rows // 2 - 35, rows // 2 + 35), (rows - 70, rows)):
        q, s = T.mx4_pack(f64(x[a:b]))
        assert np.array_equal(m.q[a:b].cpu().numpy(), q) and np.array_equal(m.scale[:, a:b].cpu().numpy(), s)
        assert np.array_equal(to_np(out[a:b]), T.mx4_unpack(q, s, cols).astype(np.float32), equal_nan=True)
    # the rows between: as calls on parts of them, which stay in the caches
    step = 40 * MIB // cols
    for a in range(0, rows, step):
        part = ma.mx4_pack(x[a:a + step])
        assert torch.equal(part.q, m.q[a:a + step]) and torch.equal(part.scale, m.scale[:, a:a + step])
        assert torch.equal(ma.mx4_unpack(part).view(torch.int16), out[a:a + step].view(torch.int16))


# a shape for each number of lanes and chunks per row
@pytest.mark.parametrize("rows,cols", [(60001, 505), (30001, 1000), (16001, 2047), (8001, 4090), (4001, 8192), (2001, 16381)])
@pytest.mark.parametrize("xd,rd,yd,held", [(BF16, BF16, None, True), (BF16, BF16, BF16, True), (BF16, F32, BF16, False), (BF16, F32, None, True), (F32, None, F32, False)])
def test_rmsnorm_past_the_caches(rows, cols, xd, rd, yd, held):
    say("rmsnorm_forward, large", rows, cols, xd, rd, yd, held)
    x, r = randn((rows, cols), 320, xd), None if rd is None else randn((rows, cols), 321, rd)
    gain = 1 + 0.3 * randn((cols,), 322)

    def call(a, b):
        n = b - a
        ck = ma.ActCheckpoint.empty(n, cols, DEV) if held else None
        out = None if yd is None else torch.empty(n, cols, dtype=yd, device=DEV)
        _, t, rstd = ma.rmsnorm_forward(x[a:b], gain, None if r is None else r[a:b], out=out, held=ck)
        return [t, rstd] + ([] if out is None else [out]) + ([ck.q, ck.scale] if held else [])
    size = x.element_size() + (0 if r is None else 2 * r.element_size()) + (0 if yd is None else 4 if yd == F32 else 2) + (1 if held else 0)
    assert rows * cols * size > 96 * MIB
    got = call(0, rows)
    # in parts that stay in the caches; pure bf16 rows go by other lanes where there are 512 or fewer
    fewest = 1 if F32 in (xd, rd, yd) else 600
    step = max(fewest, 30 * MIB // (size * cols))
    assert step * cols * size <= 96 * MIB
    for a in range(0, rows, step):
        b = min(a + step, rows)
        a = b - step
        assert all(torch.equal(p, q[a:b]) for p, q in zip(call(a, b), got))
    for a, b in ((0, 20), (rows - 20, rows)):
        y, t, rstd = T.rmsnorm_forward(f64(x[a:b]), f64(gain), None if r is None else to_np(r[a:b]), bf16_stream=rd == BF16)
        assert np.array_equal(f64(got[0][a:b]), t)
        if yd is not None:
            close(got[2][a:b], y, rms_y_tol(None, None, None, y), yd)
