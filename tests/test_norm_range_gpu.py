"""moe_add_rmsnorm where the row's sum of squares leaves fp32's range, on both sides."""
import pytest
import torch

import token_dispatch_moe_b200 as moe

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("d", [8, 128, 1024, 2880])
def test_sum_of_squares_out_of_range(d):
    x = torch.full((4, d), 1.0, device=DEV)
    x[1] = 3e19                              # 9e38: past the largest number
    x[2] = 1e-24                             # 1e-48: below the smallest, so 0
    x[3] = 1e18 / d ** 0.5                   # just inside
    x = x.to(torch.bfloat16)
    gain = torch.full((d,), 2.0, dtype=torch.bfloat16, device=DEV)
    y, mx = torch.empty_like(x), moe.MxRows.empty((4,), d, moe.MOE_MX_E4M3)
    moe.moe_add_rmsnorm(x, None, gain, 1e-6, y=y, mx=mx)
    y = y.float().cpu()
    assert (y[0] == 2.0).all() and not y[1].any() and (y[3] == 2.0).all()
    # eps alone is left: 1e-24 * 2 / sqrt(1e-6), within half a bf16 step and the norm's own 2^-18
    want = x[2].double().cpu() * 2.0 / 1e-6 ** 0.5
    assert ((y[2].double() - want).abs() <= want * (2.0 ** -8 + 2.0 ** -18)).all()
    back = torch.empty_like(x)
    moe.moe_mx_dequantize(mx, back)
    assert not back[1].any() and (back[0] == 2.0).all()
