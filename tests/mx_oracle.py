"""Microscaled rows and the operators on them in 64 bits, on the CPU, from their
definitions (numpy and exact arithmetic; nothing of the library).

Bounds.  fmt_half(fmt): the most by which rounding moves a scaled element v:
half a step, relative (eps/2: e4m3 2^-4, e2m1 2^-2) above the smallest normal
number, absolute (e4m3 2^-10, e2m1 2^-2) below.  product_bound: every product of
two elements and two powers of two is exact in fp32; the tensor core adds 32 of
them and the accumulator at a time, each term cut to 24 bits of the largest
partial sum, so a step loses at most 2 * 2^-23 of sum|x w|, and the terms'
own alignment as much again: 2^-21 * (K/32 + 1) * sum|x w| in all.
"""
import numpy as np

E4M3, E2M1 = 0, 1
_E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def _e4m3_table():
    t = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        v = m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        if e == 15 and m == 7:
            v = np.nan
        t[c] = -v if c & 128 else v
    return t


_E4M3 = _e4m3_table()


def padded(K):
    return -(-K // 128) * 128


def scale_bytes(K):
    return -(-(padded(K) // 32) // 16) * 16


def elements(q, fmt):
    if fmt == E4M3:
        return _E4M3[q]
    code = np.stack((q & 15, q >> 4), -1).reshape(*q.shape[:-1], -1)
    return np.where(code & 8, -1.0, 1.0) * _E2M1[code & 7]


def scale_values(b):
    b = b.astype(np.int64)
    return np.where(b == 255, np.nan, np.ldexp(1.0, np.minimum(b, 254) - 127))


def dequantize(q, scales, K, fmt):
    v = elements(q, fmt)
    s = np.repeat(scale_values(scales[..., :v.shape[-1] // 32]), 32, axis=-1)
    return (v * s)[..., :K]


def _nearest(v, fmt):
    """Codes of |v| (at most the format's largest): nearest, ties to the even code."""
    grid = _E2M1 if fmt == E2M1 else _E4M3[:127]
    hi = np.clip(np.searchsorted(grid, v), 1, len(grid) - 1)
    lo = hi - 1
    dl, dh = v - grid[lo], grid[hi] - v
    return np.where((dh < dl) | ((dh == dl) & (hi % 2 == 0)), hi, lo)


def scale_byte(amax, fmt):
    """Smallest b >= 0 with amax <= largest * 2^(b - 127); 255 for no number."""
    largest = 448.0 if fmt == E4M3 else 6.0
    steps = largest * np.ldexp(1.0, np.arange(0, 255) - 127)
    b = np.searchsorted(steps, np.where(np.isfinite(amax), amax, 0.0))
    return np.where(np.isfinite(amax), np.minimum(b, 254), 255).astype(np.uint8)


def quantize(x, fmt):
    """(q, scales) with all padding, of rows [rows, K] in 64 bits."""
    rows, K = x.shape
    v = np.zeros((rows, padded(K)))
    v[:, :K] = x
    blocks = v.reshape(rows, -1, 32)
    amax = np.abs(blocks).max(2)          # NaN wins in numpy's max
    b = scale_byte(amax, fmt)
    bad = b == 255
    scaled = np.where(bad[:, :, None], 0.0, blocks) / np.ldexp(1.0, np.where(bad, 127, b).astype(int) - 127)[:, :, None]
    code = _nearest(np.abs(scaled), fmt)
    sign = np.signbit(scaled) & ~bad[:, :, None]
    if fmt == E4M3:
        q = (code | (sign << 7)).astype(np.uint8).reshape(rows, -1)
    else:
        c = (code | (sign << 3)).astype(np.uint8).reshape(rows, -1)
        q = c[:, 0::2] | (c[:, 1::2] << 4)
    s = np.zeros((rows, scale_bytes(K)), dtype=np.uint8)
    s[:, :b.shape[1]] = b
    return q, s


def fmt_half(v, scale, fmt):
    """Bound of the rounding of value v in a block of the given scale (see above)."""
    rel, least = (2.0 ** -4, 2.0 ** -10) if fmt == E4M3 else (2.0 ** -2, 2.0 ** -2)
    return np.maximum(rel * np.abs(v), least * scale)


def product_bound(K, absum):
    return 2.0 ** -21 * (K / 32 + 1) * absum


def activate(g, u, oai):
    with np.errstate(over="ignore"):   # a gate far below zero: its limit, 0
        if oai:
            g, u = np.minimum(g, 7.0), np.clip(u, -7.0, 7.0)
            return g / (1.0 + np.exp(-1.702 * g)) * (u + 1.0)
        return g / (1.0 + np.exp(-g)) * u


def gate_up(x, w1, w3, b1, b3, oai, K):
    """(h, bound of h before its rounding) of one expert's rows x [n, K], w1, w3 [F, K]."""
    g, u = x @ w1.T + b1, x @ w3.T + b3
    # the bias' addition rounds once more
    dg = product_bound(K, np.abs(x) @ np.abs(w1).T) + 2.0 ** -23 * np.abs(g)
    du = product_bound(K, np.abs(x) @ np.abs(w3).T) + 2.0 ** -23 * np.abs(u)
    h = activate(g, u, oai)
    # slopes: x sigmoid(a x) rises by at most 1.1 for a >= 1; the fast exponential and quotient
    # are within 2^-20 + 2^-22 |a x| relative
    fast = (2.0 ** -20 + 2.0 ** -22 * 1.702 * np.abs(g)) * np.abs(h)
    gate = np.abs(np.minimum(g, 7.0) if oai else g)
    return h, 1.1 * (np.abs(u) + 1.0) * dg + (gate + dg) * du + fast


def down(x, w2, b2, K):
    y = x @ w2.T + b2
    return y, product_bound(K, np.abs(x) @ np.abs(w2).T) + 2.0 ** -23 * np.abs(y) + 2.0 ** -8 * np.abs(y)


def rmsnorm(x, r, gain, eps, bf16):
    """(h, y before its rounding); bf16 rounds an array to bf16."""
    h = x if r is None else bf16(x + r)
    return h, h / np.sqrt((h * h).mean(1, keepdims=True) + eps) * gain
