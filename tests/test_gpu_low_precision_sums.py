"""The sums of the product of 8-bit rows with 4-bit weights: products beside much larger ones are kept for results in
bf16 as for those in fp32."""
import pytest
import torch

import adamw_optimizer_step_amd as ma
from gpu_util import need_gpu, say
from test_gpu_low_precision import FORMS, beside_large
from test_gpu_ops import BF16, DEV, F32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


@pytest.mark.parametrize("rows,outs,ins", [(1, 40, 300), (3, 17, 100), (20, 64, 4000), (60, 64, 700), (200, 300, 1030)] + [f[:3] for f in FORMS])
def test_bf16_results_are_the_exact_sums_rounded_once(rows, outs, ins):
    """All sums are multiples of 2^-10 below 2^14, so exact in fp32 in any order: the bf16 result is their rounding."""
    say("mx4_matmul to bf16, small beside large", rows, outs, ins)
    x, w, xv, wv = beside_large(rows, outs, ins)
    want = torch.mm(xv, wv.t())
    assert bool((want.float().double() == want).all())
    assert torch.equal(ma.mx4_matmul(x, w), want.float().bfloat16())
    assert torch.equal(ma.mx4_matmul(x, w, out=torch.full((rows, outs), 0.25, dtype=BF16, device=DEV), accumulate=True), (want + 0.25).float().bfloat16())


@pytest.mark.parametrize("rows,outs", [(1, 40), (20, 64), (60, 200), (300, 520), (1300, 1700), (6000, 9001)])
@pytest.mark.parametrize("yd", [BF16, F32])
def test_small_products_remain_where_large_ones_cancel(rows, outs, yd):
    """448 * 6 - 448 * 6 + 14 * 0.234375 * 0.5, the two large products in different groups of 8: 1.640625, exact in bf16."""
    say("mx4_matmul, large ones cancel", rows, outs, yd)
    xv, wv = torch.zeros(256, device=DEV), torch.zeros(256, device=DEV)
    xv[128:144], wv[128:144] = 0.234375, 0.5
    xv[128], xv[136], wv[128], wv[136] = 448.0, -448.0, 6.0, 6.0
    x, w = ma.act_pack(xv.expand(rows, 256).contiguous()), ma.mx4_pack(wv.expand(outs, 256).contiguous())
    assert torch.equal(ma.act_unpack(x, dtype=F32)[0], xv) and torch.equal(ma.mx4_unpack(w, dtype=F32)[0], wv)
    assert torch.equal(ma.mx4_matmul(x, w, dtype=yd), torch.full((rows, outs), 1.640625, dtype=yd, device=DEV))
