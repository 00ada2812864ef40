"""moe_expert_gate_up_mx and moe_expert_down_mx against their 64-bit definition on
the same MX operands (bounds: mx_oracle)."""
import numpy as np
import pytest
import torch

import mx_oracle as mo
import token_dispatch_moe_b200 as moe

pytestmark = pytest.mark.gpu
DEV = "cuda"
E4, E2 = moe.MOE_MX_E4M3, moe.MOE_MX_E2M1
SWIGLU, OAI = moe.MOE_ACT_SWIGLU, moe.MOE_ACT_SWIGLU_OAI


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def randn(shape, seed, std=1.0):
    return torch.randn(shape, generator=gen(seed), device=DEV) * std


def mx_of(x, fmt):
    mx = moe.MxRows.empty(x.shape[:-1], x.shape[-1], fmt)
    moe.moe_mx_quantize(x.to(torch.bfloat16), mx)
    return mx


def filled(lead, K, fmt, byte=0xA5):
    return moe.MxRows(*(torch.full_like(t, byte) for t in moe.MxRows.empty(lead, K, fmt)[:2]), K, fmt)


def f64(mx, at=slice(None)):
    return mo.dequantize(mx.q[at].cpu().numpy(), mx.scales[at].cpu().numpy(), mx.K, mx.format)


def blocks(counts, first=0):
    off = np.concatenate(([0], np.cumsum(counts))) + first
    return off, torch.tensor(off, dtype=torch.int32, device=DEV)


def check_h(h, want, bound, at):
    """MX rows `at` of h against their values before rounding."""
    F = want.shape[1]
    q, s = h.q[at].cpu().numpy(), h.scales[at].cpu().numpy()
    nb = mo.padded(F) // 32
    pad = np.zeros((want.shape[0], mo.padded(F)))
    pad[:, :F] = np.abs(want)
    lo, hi = pad.copy(), pad.copy()
    lo[:, :F] = np.maximum(lo[:, :F] - bound, 0)
    hi[:, :F] += bound
    b_lo = mo.scale_byte(lo.reshape(len(pad), nb, 32).max(2), h.format)
    b_hi = mo.scale_byte(hi.reshape(len(pad), nb, 32).max(2), h.format)
    assert ((s[:, :nb] >= b_lo) & (s[:, :nb] <= b_hi)).all()
    assert not s[:, nb:].any()
    v = mo.dequantize(q, s, mo.padded(F), h.format)
    assert not v[:, F:].any()
    scale = np.repeat(mo.scale_values(s[:, :nb]), 32, axis=1)[:, :F]
    # the kernel rounds its own h, within `bound` of want
    err = np.abs(v[:, :F] - want)
    lim = mo.fmt_half(np.abs(want) + bound, scale, h.format) + bound
    assert (err <= lim).all(), (err / lim).max()


CASES = [
    # counts, d, F, x format, w format, h format, act, bias, first row
    ([1], 128, 64, E4, E2, E4, SWIGLU, False, 0),
    ([3], 128, 32, E4, E4, E4, SWIGLU, False, 0),
    ([8, 0, 1], 256, 128, E4, E2, E4, OAI, True, 0),
    ([0, 0, 5, 0], 64, 8, E2, E2, E2, SWIGLU, True, 0),
    ([1, 1, 1, 1], 2880, 2880, E4, E2, E4, OAI, True, 0),        # a decoded token of gpt-oss
    ([7, 9, 0, 16, 33, 2], 136, 72, E4, E2, E2, OAI, True, 3),
    ([31, 32, 33, 63, 65], 392, 200, E2, E4, E4, SWIGLU, False, 5),
    ([127, 129, 128], 520, 264, E4, E2, E4, OAI, True, 0),
    ([223, 225, 0, 224, 449], 640, 328, E4, E2, E4, SWIGLU, True, 1),
    ([700, 3, 500], 1288, 96, E4, E4, E4, SWIGLU, False, 0),     # several parts a block
    ([40] * 50, 256, 128, E4, E2, E4, OAI, True, 0),             # more tiles than SMs
    ([90, 11], 2048, 768, E4, E2, E4, SWIGLU, False, 0),         # the qwen3 expert
    ([30, 35, 31], 264, 72, E4, E2, E4, SWIGLU, True, 0),        # token tiles of 48, one CTA
    ([64, 50, 78, 81], 264, 72, E2, E2, E4, OAI, False, 2),      # 80, pairs from here
    ([95, 65, 97, 63], 136, 200, E4, E2, E2, SWIGLU, True, 0),   # 96
    ([180, 150, 210, 211], 136, 200, E4, E4, E4, OAI, True, 0),  # 208
    ([350, 300, 1, 0, 1020], 136, 72, E4, E2, E4, SWIGLU, True, 7),  # two parts and more
    ([2, 0, 1, 4] * 32, 72, 40, E4, E2, E4, OAI, True, 0),       # 128 experts of few rows
]


def ident(c):
    n = len(c[0])
    return f"{n}x{max(c[0])}-" + "-".join(map(str, c[1:]))


@pytest.mark.parametrize("case", CASES, ids=ident)
def test_gate_up(case):
    counts, d, F, xf, wf, hf, act, bias, first = case
    E = len(counts)
    off, offsets = blocks(counts, first)
    rows = int(off[-1]) + 9                       # rows behind the last block
    x = randn((rows, d), 1) * torch.exp(randn((rows, 1), 2))
    xs = mx_of(x, xf)
    w1, w3 = mx_of(randn((E, F, d), 3, d ** -0.5), wf), mx_of(randn((E, F, d), 4, d ** -0.5), wf)
    b1, b3 = (randn((E, F), 5, 0.5), randn((E, F), 6, 0.5)) if bias else (None, None)
    h = filled((rows,), F, hf)
    st = torch.zeros((1,), dtype=torch.int32, device=DEV)
    moe.moe_expert_gate_up_mx(xs, offsets, w1, w3, h, b1, b3, act, st)
    torch.cuda.synchronize()
    assert st.item() == 0
    for e in range(E):
        at = slice(int(off[e]), int(off[e + 1]))
        if at.start == at.stop:
            continue
        bb = [t[e].double().cpu().numpy() if t is not None else 0.0 for t in (b1, b3)]
        want, bound = mo.gate_up(f64(xs, at), f64(w1, e), f64(w3, e), *bb, act == OAI, d)
        check_h(h, want, bound, at)
    for t in (h.q, h.scales):                     # rows outside the blocks: as they were
        assert (t[:first] == 0xA5).all() and (t[int(off[-1]):] == 0xA5).all()


@pytest.mark.parametrize("case", CASES, ids=ident)
def test_down(case):
    counts, d, F, hf, wf, _, _, bias, first = case
    E = len(counts)
    off, offsets = blocks(counts, first)
    rows = int(off[-1]) + 9
    h = mx_of(randn((rows, F), 1) * torch.exp(randn((rows, 1), 2)), hf)
    w2 = mx_of(randn((E, d, F), 3, F ** -0.5), wf)
    b2 = randn((E, d), 5, 0.5) if bias else None
    y = torch.full((rows, d), 9.0, dtype=torch.bfloat16, device=DEV)
    st = torch.zeros((1,), dtype=torch.int32, device=DEV)
    moe.moe_expert_down_mx(h, offsets, w2, y, b2, st)
    torch.cuda.synchronize()
    assert st.item() == 0
    for e in range(E):
        at = slice(int(off[e]), int(off[e + 1]))
        if at.start == at.stop:
            continue
        want, bound = mo.down(f64(h, at), f64(w2, e), b2[e].double().cpu().numpy() if bias else 0.0, F)
        err = np.abs(y[at].double().cpu().numpy() - want)
        assert (err <= bound).all(), (err / bound).max()
    assert (y[:first] == 9.0).all() and (y[int(off[-1]):] == 9.0).all()


@pytest.mark.parametrize("fmt", [E4, E2])
def test_integer_products_are_exact(fmt):
    """Small integers and powers of two as scales: every sum is exact, so every bit is known.
    A different scale in each block and row shows a scale applied to the wrong place."""
    E, d, F, counts = 3, 384, 136, [70, 1, 230]
    off, offsets = blocks(counts)
    rows = int(off[-1])
    g = np.random.default_rng(1)

    def ints(*lead, K):
        code = g.integers(0, 16, (*lead, mo.padded(K)), dtype=np.uint8)
        code[..., 0:6] &= 7
        if fmt == E2:
            q = code[..., 0::2] | (code[..., 1::2] << 4)
        else:  # the same values in e4m3
            table = np.array([0x00, 0x30, 0x38, 0x3C, 0x40, 0x44, 0x48, 0x4C], dtype=np.uint8)
            q = table[code & 7] | ((code & 8) << 4)
        s = np.zeros((*lead, mo.scale_bytes(K)), dtype=np.uint8)
        s[..., :mo.padded(K) // 32] = g.integers(125, 130, (*lead, mo.padded(K) // 32))
        return moe.MxRows(torch.from_numpy(q).to(DEV), torch.from_numpy(s).to(DEV), K, fmt)

    h, w2 = ints(rows, K=F), ints(E, d, K=F)
    # padding columns of the operands are zeros
    for t in (h, w2):
        t.q[..., (F if fmt == E4 else F // 2):] = 0
    y = torch.empty((rows, d), dtype=torch.bfloat16, device=DEV)
    moe.moe_expert_down_mx(h, offsets, w2, y)
    for e in range(E):
        at = slice(int(off[e]), int(off[e + 1]))
        want = f64(h, at) @ f64(w2, e).T
        assert torch.equal(y[at].cpu(), torch.from_numpy(want).to(torch.float32).to(torch.bfloat16))


@pytest.mark.parametrize("off", [[0, 40, 30, 64], [-1, 10, 20, 64], [0, 10, 20, 65], [5, 4, 4, 4]])
def test_bad_offsets_are_reported(off):
    E, d, F, rows = 3, 128, 64, 64
    offsets = torch.tensor(off, dtype=torch.int32, device=DEV)
    xs, w = mx_of(randn((rows, d), 1), E4), mx_of(randn((E, F, d), 2), E2)
    h = filled((rows,), F, E4)
    st = torch.zeros((1,), dtype=torch.int32, device=DEV)
    moe.moe_expert_gate_up_mx(xs, offsets, w, w, h, d_status=st)
    torch.cuda.synchronize()
    assert st.item() == moe.MOE_ERR_DEVICE_INDEX
    assert (h.q == 0xA5).all() and (h.scales == 0xA5).all()


@pytest.mark.parametrize("act", [SWIGLU, OAI])
def test_not_a_number_stays_in_its_row(act):
    E, d, F, counts = 2, 256, 64, [20, 21]
    off, offsets = blocks(counts)
    rows = int(off[-1])
    x = randn((rows, d), 1)
    x[7, 100] = float("nan")
    x[20, 3] = float("inf")
    w = mx_of(randn((E, F, d), 2, 0.1), E2)
    h = filled((rows,), F, E4)
    moe.moe_expert_gate_up_mx(mx_of(x, E4), offsets, w, w, h, act=act)
    nan = (h.scales[:, :2] == 255).any(1).cpu()
    assert nan[7] and nan[20] and nan.sum() == 2
    w2 = mx_of(randn((E, d, F), 3, 0.1), E2)
    y = torch.empty((rows, d), dtype=torch.bfloat16, device=DEV)
    moe.moe_expert_down_mx(h, offsets, w2, y)
    nan = torch.isnan(y).cpu()
    assert nan[7].all() and nan[20].all() and nan.any(1).sum() == 2


@pytest.mark.parametrize("act", [SWIGLU, OAI])
def test_gates_far_out(act):
    """Gates and ups far beyond the exponential's range, on both sides: 0, the limit or the
    product, never NaN."""
    E, d, F, rows = 1, 32, 32, 16
    x = torch.zeros((rows, d), device=DEV)
    x[:, 0] = torch.tensor([0, 1e-3, 1, 20, 90, 130, 300, 1e4, 0, -1e-3, -1, -20, -90, -130, -300, -1e4], device=DEV)
    w1, w3 = torch.zeros((E, F, d), device=DEV), torch.zeros((E, F, d), device=DEV)
    w1[:, :, 0] = torch.linspace(0.5, 2, F, device=DEV)
    w3[:, :, 0] = torch.linspace(-1, 1, F, device=DEV)
    off, offsets = blocks([rows])
    xs, m1, m3 = mx_of(x, E4), mx_of(w1, E4), mx_of(w3, E4)
    h = filled((rows,), F, E4)
    moe.moe_expert_gate_up_mx(xs, offsets, m1, m3, h, act=act)
    want, bound = mo.gate_up(f64(xs), f64(m1, 0), f64(m3, 0), 0.0, 0.0, act == OAI, d)
    assert np.isfinite(want).all()
    check_h(h, want, bound, slice(0, rows))


def test_most_experts():
    """4096 experts, most of them without a row."""
    E, d, F = 4096, 64, 32
    counts = (np.arange(E) % 37 == 5).astype(int) * (1 + np.arange(E) % 3)
    off, offsets = blocks(counts)
    rows = int(off[-1])
    xs = mx_of(randn((rows, d), 1), E4)
    w1, w2 = mx_of(randn((E, F, d), 2, 0.1), E2), mx_of(randn((E, d, F), 3, 0.1), E2)
    h, y = filled((rows,), F, E4), torch.empty((rows, d), dtype=torch.bfloat16, device=DEV)
    st = torch.zeros((1,), dtype=torch.int32, device=DEV)
    moe.moe_expert_gate_up_mx(xs, offsets, w1, w1, h, d_status=st)
    moe.moe_expert_down_mx(h, offsets, w2, y, d_status=st)
    torch.cuda.synchronize()
    assert st.item() == 0
    for e in np.nonzero(counts)[0]:
        at = slice(int(off[e]), int(off[e + 1]))
        want, bound = mo.gate_up(f64(xs, at), f64(w1, e), f64(w1, e), 0.0, 0.0, False, d)
        check_h(h, want, bound, at)
        want, bound = mo.down(f64(h, at), f64(w2, e), 0.0, F)
        assert (np.abs(y[at].double().cpu().numpy() - want) <= bound).all()


def test_rows_past_32_bits():
    """Results of more than 2^32 bytes: the last rows are right and in their place."""
    E, d, F = 2, 40, 4104
    rows = (1 << 20) + 77
    off, offsets = blocks([5, rows - 5])
    xs = moe.MxRows(*(torch.zeros_like(t) for t in moe.MxRows.empty((rows,), d, E4)[:2]), d, E4)
    tail = mx_of(randn((9, d), 1), E4)
    xs.q[-9:], xs.scales[-9:] = tail.q, tail.scales
    w1 = mx_of(randn((E, F, d), 2, 0.2), E2)
    h = moe.MxRows.empty((rows,), F, E4)
    moe.moe_expert_gate_up_mx(xs, offsets, w1, w1, h)
    want, bound = mo.gate_up(f64(tail), f64(w1, 1), f64(w1, 1), 0.0, 0.0, False, d)
    check_h(h, want, bound, slice(rows - 9, rows))
    assert not h.q[5:rows - 9].any()
    del h
    w2 = mx_of(randn((E, F, d), 3, 0.2), E2)          # as a down matrix: d inputs, F outputs
    y = torch.empty((rows, F), dtype=torch.bfloat16, device=DEV)
    moe.moe_expert_down_mx(xs, offsets, w2, y)
    want, bound = mo.down(f64(tail), f64(w2, 1), 0.0, d)
    assert (np.abs(y[-9:].double().cpu().numpy() - want) <= bound).all()
    assert not y[5:-9].any()


def test_no_rows():
    E, d, F = 2, 64, 32
    w1, w2 = mx_of(randn((E, F, d), 1), E2), mx_of(randn((E, d, F), 1), E2)
    offsets = torch.zeros((E + 1,), dtype=torch.int32, device=DEV)
    h = filled((5,), F, E4)
    moe.moe_expert_gate_up_mx(mx_of(randn((5, d), 2), E4), offsets, w1, w1, h)   # empty blocks
    assert (h.q == 0xA5).all()
    h0, x0 = moe.MxRows.empty((0,), F, E4), moe.MxRows.empty((0,), d, E4)
    moe.moe_expert_gate_up_mx(x0, offsets, w1, w1, h0)                          # no rows at all
    moe.moe_expert_down_mx(h0, offsets, w2, torch.empty((0, d), dtype=torch.bfloat16, device=DEV))


def test_refusals():
    E, d, F, rows = 2, 128, 64, 16
    offsets = torch.tensor([0, 8, 16], dtype=torch.int32, device=DEV)
    xs, w1 = mx_of(randn((rows, d), 1), E4), mx_of(randn((E, F, d), 2), E2)
    h = moe.MxRows.empty((rows,), F, E4)
    with pytest.raises(moe.MoeError):
        moe.moe_expert_gate_up_mx(xs, offsets, w1, w1, h, act=5)
    with pytest.raises(ValueError):     # weights of two formats
        moe.moe_expert_gate_up_mx(xs, offsets, w1, mx_of(randn((E, F, d), 2), E4), h)
    with pytest.raises(ValueError):     # rows of another width
        moe.moe_expert_gate_up_mx(mx_of(randn((rows, 256), 1), E4), offsets, w1, w1, h)
    with pytest.raises(ValueError):     # offsets of another expert count
        moe.moe_expert_gate_up_mx(xs, offsets[:2].contiguous(), w1, w1, h)
    with pytest.raises(ValueError):     # q of the other format's width
        moe.moe_expert_gate_up_mx(xs._replace(format=E2), offsets, w1, w1, h)
    with pytest.raises(TypeError):
        moe.moe_expert_down_mx(h, offsets, mx_of(randn((E, d, F), 3), E2), torch.empty((rows, d), device=DEV))
    with pytest.raises(moe.MoeError):   # rows that begin 16 bytes into their storage
        raw = torch.zeros((rows * 128 + 32,), dtype=torch.uint8, device=DEV)[16:16 + rows * 128]
        moe.moe_expert_gate_up_mx(xs._replace(q=raw.view(rows, 128)), offsets, w1, w1, h)
