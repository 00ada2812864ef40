"""moe_expert_gate_up_mx at the ends of fp32's range: gates, ups and results that no network
reaches but finite operands can."""
import numpy as np
import pytest
import torch

import mx_oracle as mo
import token_dispatch_moe_b200 as moe
from test_expert_ffn_mx_gpu import DEV, E4, OAI, SWIGLU, blocks, check_h, filled, mx_of

pytestmark = pytest.mark.gpu
FLT_MAX = float(np.finfo(np.float32).max)


def of_biases(g, u, act, fmt=E4):
    """h of rows whose products are 0: gate and up are the biases g, u [F] (fp32, exactly)."""
    F, d, rows = len(g), 32, 3
    _, offsets = blocks([rows])
    zero = lambda *lead: mx_of(torch.zeros((*lead, d), device=DEV), E4)
    b1, b3 = (torch.tensor(np.asarray(v, dtype=np.float32)[None], device=DEV) for v in (g, u))
    h = filled((rows,), F, fmt)
    st = torch.zeros((1,), dtype=torch.int32, device=DEV)
    moe.moe_expert_gate_up_mx(zero(rows), offsets, zero(1, F), zero(1, F), h, b1, b3, act, st)
    torch.cuda.synchronize()
    assert st.item() == 0
    b1, b3 = (np.repeat(t.double().cpu().numpy(), rows, 0) for t in (b1, b3))
    return h, b1, b3


@pytest.mark.parametrize("act", [SWIGLU, OAI])
@pytest.mark.parametrize("fmt", [moe.MOE_MX_E4M3, moe.MOE_MX_E2M1])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_gates_at_the_end_of_the_range(sign, fmt, act):
    """log2(e) times the gate passes fp32's largest number from 2.36e38 on: the value is still
    gate times up (SwiGLU), the limit's (clamped), or 0."""
    g = sign * np.array([2.0e38, 2.35e38, 2.3584e38, 2.36e38, 2.3647e38, 2.4e38, 3.0e38, FLT_MAX] * 12)
    u = np.concatenate((np.linspace(0.25, 0.99, 32), np.linspace(-3e-38, 3e-38, 32), np.linspace(-0.5, 0.5, 32)))
    h, g, u = of_biases(g, u, act, fmt)
    want = mo.activate(g, u, act == OAI)
    assert np.isfinite(want).all()
    # The exponential is 0 (or, clamped, of 11.9 at most: as the other tests bound it); a
    # reciprocal within 2^-23, two sums and two products within 2^-24 each: under 2^-21, and
    # 2^-20 + 2^-22 * 11.9 for the clamped form.  On the far negative side the value is 0.
    rel = 2.0 ** -20 + 2.0 ** -22 * 11.9 if act == OAI else 2.0 ** -21
    check_h(h, want, rel * np.abs(want), slice(0, 3))


@pytest.mark.parametrize("act", [SWIGLU, OAI])
@pytest.mark.parametrize("up", [1.0, 7.0, 1e38])
def test_gates_whose_sigmoid_counts_as_zero(up, act):
    """Gates from -40 to -200 with ups of one size: a sigmoid below 2^-126 may count as 0."""
    g = -np.linspace(40, 200, 96)
    h, g, u = of_biases(g, np.full(96, up), act)
    want = mo.activate(g, u, act == OAI)
    factor = np.clip(u, -7.0, 7.0) + 1.0 if act == OAI else u
    # what counts as 0, and the exponential's bound as in the other tests
    bound = np.abs(g * factor) * 2.0 ** -126 + np.abs(want) * (2.0 ** -20 + 2.0 ** -22 * 1.702 * np.abs(g))
    check_h(h, want, bound, slice(0, 3))
