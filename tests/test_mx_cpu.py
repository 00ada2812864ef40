"""The MX entry points without a GPU: row lengths, and refusals that come before any
CUDA call (the pointers here are never read)."""
import ctypes

import pytest
import torch

import mx_oracle as mo
import token_dispatch_moe_b200 as moe
from token_dispatch_moe_b200 import build as build_mod

P = ctypes.c_void_p
OK, BAD, BIG = moe.MOE_OK, moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_UNSUPPORTED
A = P(4096)          # aligned for everything


@pytest.fixture(scope="module")
def lib():
    return moe.load_library(build_mod.build())


def test_row_bytes(lib):
    for K in (8, 120, 128, 136, 2056, 2880, 7168, 262144):
        assert moe.moe_mx_row_bytes(K, moe.MOE_MX_E4M3) == (mo.padded(K), mo.scale_bytes(K))
        assert moe.moe_mx_row_bytes(K, moe.MOE_MX_E2M1) == (mo.padded(K) // 2, mo.scale_bytes(K))
    assert moe.moe_mx_row_bytes(2880, moe.MOE_MX_E2M1) == (1472, 96)
    for K, fmt in ((0, 0), (-8, 0), (12, 0), (64, 2), (64, -1), (262152, 0)):
        with pytest.raises(moe.MoeError):
            moe.moe_mx_row_bytes(K, fmt)


def test_rows_refusals(lib):
    for rows, K, fmt, x, q, s, want in (
            (4, 64, 2, A, A, A, BAD), (4, 12, 0, A, A, A, BAD), (4, 0, 0, A, A, A, BAD),
            (-1, 64, 0, A, A, A, BAD), (4, 64, 0, None, A, A, BAD), (4, 64, 0, A, None, A, BAD),
            (4, 64, 0, A, A, None, BAD), (4, 64, 0, P(4104), A, A, BAD),
            (4, 64, 0, A, P(4112), A, BAD), (4, 64, 0, A, A, P(4104), BAD),
            (4, 262152, 0, A, A, A, BIG), (1 << 31, 64, 0, A, A, A, BIG),
            (0, 64, 0, None, None, None, OK)):
        assert lib.moe_mx_quantize(x, rows, K, fmt, q, s, None) == want
        assert lib.moe_mx_dequantize(q, s, rows, K, fmt, x, None) == want


def norm(lib, x=A, r=A, g=A, eps=1e-5, T=4, d=64, h=A, y=P(8192), fmt=0, q=A, s=A):
    return lib.moe_add_rmsnorm(x, r, g, eps, T, d, h, y, fmt, q, s, None)


def test_norm_refusals(lib):
    assert norm(lib, T=0) == OK
    for kw in (dict(T=-1), dict(d=12), dict(d=0), dict(eps=-1.0), dict(eps=float("nan")),
               dict(fmt=3), dict(s=None), dict(q=None), dict(x=None), dict(g=None),
               dict(h=None, y=None, q=None, s=None), dict(x=P(4104)), dict(r=P(4104)),
               dict(g=P(4104)), dict(y=P(8192), h=P(8192)), dict(h=P(4104)), dict(y=P(4104)), dict(q=P(4112)), dict(s=P(4104))):
        assert norm(lib, **kw) == BAD, kw
    assert norm(lib, d=16392) == BIG
    assert norm(lib, T=1 << 31) == BIG


def gate_up(lib, x=A, xs=A, xf=0, off=A, w1=A, w1s=A, w3=A, w3s=A, wf=1, b1=None, b3=None, E=4,
            d=64, F=32, rows=8, act=0, h=A, hs=A, hf=0):
    return lib.moe_expert_gate_up_mx(x, xs, xf, off, w1, w1s, w3, w3s, wf, b1, b3, E, d, F, rows,
                                     act, h, hs, hf, None, None)


def down(lib, x=A, xs=A, xf=0, off=A, w=A, ws=A, wf=1, b=None, E=4, d=64, F=32, rows=8, y=A):
    return lib.moe_expert_down_mx(x, xs, xf, off, w, ws, wf, b, E, d, F, rows, y, None, None)


def test_expert_refusals(lib):
    assert gate_up(lib, rows=0) == OK and down(lib, rows=0) == OK
    both = (dict(E=0), dict(E=4097), dict(d=12), dict(F=12), dict(d=0), dict(F=0), dict(rows=-1),
            dict(xf=2), dict(wf=-1), dict(x=None), dict(xs=None), dict(off=None), dict(x=P(4112)),
            dict(xs=P(4104)))
    for kw in both + (dict(act=2), dict(hf=2), dict(w1=None), dict(w1s=None), dict(w3=None),
                      dict(w3s=None), dict(h=None), dict(hs=None), dict(w1=P(4112)),
                      dict(w3s=P(4104)), dict(h=P(4112)), dict(b1=P(4100)), dict(b3=P(4100))):
        assert gate_up(lib, **kw) == BAD, kw
    for kw in both + (dict(w=None), dict(ws=None), dict(y=None), dict(w=P(4112)), dict(y=P(4104)),
                      dict(b=P(4100))):
        assert down(lib, **kw) == BAD, kw
    for f in (gate_up, down):
        assert f(lib, rows=(1 << 31) - 1) == BIG
        assert f(lib, d=262152) == BIG


def test_binding_refuses_host_tensors(lib):
    """Wrong types, and tensors that are not on the GPU, before any call."""
    x = torch.zeros((4, 64), dtype=torch.bfloat16)
    mx = moe.MxRows(torch.zeros((4, 128), dtype=torch.uint8),
                    torch.zeros((4, 16), dtype=torch.uint8), 64, moe.MOE_MX_E4M3)
    with pytest.raises(ValueError, match="CUDA"):
        moe.moe_mx_quantize(x, mx)
    with pytest.raises(TypeError):
        moe.moe_add_rmsnorm(x.float(), None, x[0], 1e-5, y=x)
    with pytest.raises(TypeError):
        moe.moe_mx_dequantize(mx._replace(q=mx.q.int()), x)
