"""moe_mx_quantize, moe_mx_dequantize (every bit) and moe_add_rmsnorm against the
64-bit definitions of mx_oracle."""
import numpy as np
import pytest
import torch

import mx_oracle as mo
import token_dispatch_moe_b200 as moe

pytestmark = pytest.mark.gpu
DEV = "cuda"
FORMATS = [moe.MOE_MX_E4M3, moe.MOE_MX_E2M1]


def bf16_of(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float64)).to(torch.float32).to(torch.bfloat16)


def f64(t):
    return t.detach().cpu().double().numpy()


def randn(shape, seed, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(torch.bfloat16)


def quantized(x, fmt):
    mx = moe.MxRows(*(torch.full_like(t, 0xA5) for t in moe.MxRows.empty((x.shape[0],), x.shape[1], fmt)[:2]),
                    x.shape[1], fmt)
    moe.moe_mx_quantize(x, mx)
    return mx


def assert_bits(mx, x):
    q, s = mo.quantize(f64(x), mx.format)
    assert np.array_equal(mx.scales.cpu().numpy(), s)
    got = mx.q.cpu().numpy()
    assert np.array_equal(got, q), np.argwhere(got != q)[:5]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("rows,K", [(1, 8), (1, 128), (3, 32), (5, 40), (257, 136), (33, 512),
                                    (7, 2056), (2, 2880), (1023, 72), (4, 7168), (1, 32768)])
def test_quantize_bits(rows, K, fmt):
    x = randn((rows, K), rows + K) * torch.exp2(torch.randint(-20, 20, (rows, 1), generator=torch.Generator().manual_seed(K)).float()).to(torch.bfloat16)
    x[:, ::7] *= 16
    mx = quantized(x.to(DEV), fmt)
    assert_bits(mx, x)
    back = torch.empty((rows, K), dtype=torch.bfloat16, device=DEV)
    moe.moe_mx_dequantize(mx, back)
    want = bf16_of(mo.dequantize(mx.q.cpu().numpy(), mx.scales.cpu().numpy(), K, fmt))
    assert torch.equal(back.cpu(), want)


@pytest.mark.parametrize("fmt", FORMATS)
def test_quantize_special_blocks(fmt):
    """Blocks of zeros, of both zeros, of subnormals, of the largest numbers, of ties and of the
    values on either side of a scale's border."""
    top = 448.0 if fmt == moe.MOE_MX_E4M3 else 6.0
    grid = mo._E4M3[:127] if fmt == moe.MOE_MX_E4M3 else mo._E2M1
    mids = (grid[1:] + grid[:-1]) / 2
    rows = [np.zeros(32), np.full(32, -0.0), np.full(32, 2.0 ** -133), np.full(32, 2.0 ** -126),
            np.full(32, float(torch.finfo(torch.bfloat16).max))]
    for s in (-3, 0, 5):
        for a in (top, top * (1 + 2.0 ** -6), top * (1 - 2.0 ** -6), 2.0 ** 8, 2.0 ** 2):
            rows.append(np.concatenate(([a * 2.0 ** s], np.linspace(-a, a, 31) * 2.0 ** s)))
    for i in range(0, len(mids), 31):
        m = mids[i:i + 31]
        rows.append(np.concatenate(([top], m, np.zeros(31 - len(m)))))
        rows.append(-rows[-1])
    x = bf16_of(np.stack(rows))
    assert_bits(quantized(x.to(DEV), fmt), x)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_quantize_not_a_number(bad, fmt):
    """A block with an infinity or NaN reads back as NaN; its neighbours do not notice."""
    x = randn((3, 96), 5)
    x[1, 40] = bad
    mx = quantized(x.to(DEV), fmt)
    assert_bits(mx, x)
    assert mx.scales[1, 1].item() == 255
    back = torch.empty((3, 96), dtype=torch.bfloat16, device=DEV)
    moe.moe_mx_dequantize(mx, back)
    nan = torch.isnan(back).cpu()
    assert nan[1, 32:64].all() and nan.sum() == 32


@pytest.mark.parametrize("fmt", FORMATS)
def test_dequantize_every_code_and_scale(fmt):
    K = 256
    q = np.tile(np.arange(256, dtype=np.uint8)[: K if fmt == moe.MOE_MX_E4M3 else K // 2], (512, 1))
    if fmt == moe.MOE_MX_E2M1:
        q[256:] += 128
    s = np.zeros((512, mo.scale_bytes(K)), dtype=np.uint8)
    s[:, :K // 32] = (np.arange(512)[:, None] + 37 * np.arange(K // 32)) % 256
    mx = moe.MxRows(torch.from_numpy(q).to(DEV), torch.from_numpy(s).to(DEV), K, fmt)
    out = torch.empty((512, K), dtype=torch.bfloat16, device=DEV)
    moe.moe_mx_dequantize(mx, out)
    with np.errstate(invalid="ignore"):
        want = mo.dequantize(q, s, K, fmt)
    got = f64(out)
    assert np.array_equal(np.isnan(got), np.isnan(want))
    ok = ~np.isnan(want)
    # elements have at most 4 bits: exact, but where bf16's least step (2^-133) is too coarse;
    # numbers past bf16's largest become infinite
    assert np.array_equal(got[ok], f64(bf16_of(want))[ok])


def test_quantize_past_32_bits():
    """More than 2^32 values: the last rows are written where they belong."""
    rows, K = (1 << 21) + 3, 2056
    x = torch.zeros((rows, K), dtype=torch.bfloat16, device=DEV)
    tail = randn((5, K), 1)
    x[-5:] = tail.to(DEV)
    mx = moe.MxRows.empty((rows,), K, moe.MOE_MX_E2M1)
    moe.moe_mx_quantize(x, mx)
    assert_bits(moe.MxRows(mx.q[-5:], mx.scales[-5:], K, moe.MOE_MX_E2M1), tail)
    x.fill_(3.0)
    moe.moe_mx_dequantize(mx, x)
    want = mo.dequantize(mx.q[-5:].cpu().numpy(), mx.scales[-5:].cpu().numpy(), K, moe.MOE_MX_E2M1)
    assert torch.equal(x[-5:].cpu(), bf16_of(want))
    assert not x[:-5].any()


NORM_CASES = [(1, 8), (1, 2880), (3, 40), (17, 128), (5, 2048), (9, 2056), (2, 7168), (4, 4104),
              (2, 16384), (300, 264), (33, 16), (19, 256), (21, 512), (9, 1024), (5, 1032)]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("T,d", NORM_CASES)
def test_norm(T, d, residual, fmt):
    x, gain = randn((T, d), d, 2.0), randn((d,), 3)
    x[:, 0] *= 50
    r = randn((T, d), 4) if residual else None
    eps = 1e-5
    dev = [t.to(DEV) if t is not None else None for t in (x, r, gain)]
    h_out, y = torch.empty_like(dev[0]), torch.empty_like(dev[0])
    mx = moe.MxRows(*(torch.full_like(t, 0xA5) for t in moe.MxRows.empty((T,), d, fmt)[:2]), d, fmt)
    moe.moe_add_rmsnorm(*dev, eps, h_out, y, mx)
    h, want = mo.rmsnorm(f64(x), None if r is None else f64(r), f64(gain), eps, lambda a: f64(bf16_of(a)))
    assert np.array_equal(f64(h_out), h)
    # fp32: d terms of the sum in a tree of at most 64 + 13 steps, halved by the root; three
    # products and the root: under 2^-24 * 48; then half a bf16 step
    bound = np.abs(want) * (2.0 ** -8 + 2.0 ** -18)
    assert (np.abs(f64(y) - want) <= bound).all()
    assert_bits(mx, y.cpu())  # the MX rows are those of y as stored
    # each output alone, and in place, gives the same bits
    only = torch.empty_like(y)
    moe.moe_add_rmsnorm(*dev, eps, y=only)
    assert torch.equal(only, y)
    mx2 = moe.MxRows.empty((T,), d, fmt)
    moe.moe_add_rmsnorm(*dev, eps, mx=mx2)
    assert torch.equal(mx2.q, mx.q) and torch.equal(mx2.scales, mx.scales)
    if residual:
        stream = dev[1].clone()
        xin = dev[0].clone()
        moe.moe_add_rmsnorm(xin, stream, dev[2], eps, residual_out=stream, y=xin)
        assert torch.equal(stream, h_out) and torch.equal(xin, y)


def test_norm_rows_of_zeros_and_nan():
    """A zero row stays zero with eps > 0; a NaN or infinite row is NaN and alone in it."""
    T, d = 4, 72
    x = randn((T, d), 1)
    x[1] = 0
    x[2, 5] = float("nan")
    x[3, 70] = float("inf")
    gain = torch.ones((d,), dtype=torch.bfloat16, device=DEV)
    y = torch.empty((T, d), dtype=torch.bfloat16, device=DEV)
    mx = moe.MxRows.empty((T,), d, moe.MOE_MX_E4M3)
    moe.moe_add_rmsnorm(x.to(DEV), None, gain, 1e-6, y=y, mx=mx)
    y = y.cpu()
    assert torch.isfinite(y[:2]).all() and not y[1].any()
    assert torch.isnan(y[2]).all() and torch.isnan(y[3, 70])
    assert not y[3, :70].any() and y[3, 71] == 0
    assert_bits(mx, y)


def test_rows_and_norm_in_a_graph_on_another_stream():
    T, d = 37, 2880
    x, r, gain = randn((T, d), 1).to(DEV), randn((T, d), 2).to(DEV), randn((d,), 3).to(DEV)
    h, y, back = (torch.empty_like(x) for _ in range(3))
    mx = moe.MxRows.empty((T,), d, moe.MOE_MX_E2M1)

    def step():
        moe.moe_add_rmsnorm(x, r, gain, 1e-5, h, y, None)
        moe.moe_mx_quantize(y, mx)
        moe.moe_mx_dequantize(mx, back)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        step()
        s.synchronize()
        with torch.cuda.graph(graph, stream=s):
            step()
    for seed in (8, 9):
        x.copy_(randn((T, d), seed))
        graph.replay()
        torch.cuda.synchronize()
        assert_bits(mx, y.cpu())
        want = bf16_of(mo.dequantize(mx.q.cpu().numpy(), mx.scales.cpu().numpy(), d, mx.format))
        assert torch.equal(back.cpu(), want)


def test_zero_rows():
    mx = moe.MxRows.empty((0,), 64, moe.MOE_MX_E4M3)
    x = torch.empty((0, 64), dtype=torch.bfloat16, device=DEV)
    moe.moe_mx_quantize(x, mx)
    moe.moe_mx_dequantize(mx, x)
    moe.moe_add_rmsnorm(x, None, torch.ones((64,), dtype=torch.bfloat16, device=DEV), 1e-5, y=x)
