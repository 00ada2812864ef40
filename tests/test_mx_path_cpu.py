"""RouterDispatch with MX activations, as far as it goes without a GPU: its buffers, and the steps
that its rows are not for."""
import dataclasses

import pytest
import torch

import token_dispatch_moe_b200 as moe
from token_dispatch_moe_b200 import build as build_mod
from token_dispatch_moe_b200.path import RouterDispatch
from token_dispatch_moe_b200.workloads import WORKLOADS


@pytest.fixture(scope="module", autouse=True)
def lib():
    return moe.load_library(build_mod.build())


def path_of(mx, ffn=True):
    wl = WORKLOADS["mixtral_tiny"].scaled(16)
    return RouterDispatch(wl.with_ffn() if ffn else wl, device="cpu", mx=mx)


@pytest.mark.parametrize("ffn", [False, True])
def test_buffers_are_those_of_the_rows(ffn):
    path = path_of(moe.MOE_MX_E4M3, ffn)
    assert path.xs is None and path.h is None          # no bf16 rows beside the MX ones
    rows = path.xs_mx.q.shape[0]
    assert path.h_mx.q.shape[0] == rows and path.y.shape == (rows, path.wl.d)
    bf16 = path_of(None, ffn)
    assert bf16.xs.shape == (rows, path.wl.d) and (bf16.h is not None) == ffn


def test_steps_of_the_other_rows_are_refused():
    w = {k: torch.zeros((1,)) for k in ("w1", "w2", "w3", "b1", "b2", "b3")}
    x = torch.zeros((16, 8), dtype=torch.bfloat16)
    path = path_of(moe.MOE_MX_E4M3)
    for step in (lambda: path.permute(x), lambda: path.expert_gate_up(w), lambda: path.expert_down(w)):
        with pytest.raises(ValueError, match="rows are MX"):
            step()
    path = path_of(None)
    for step in (lambda: path.norm(x, None, x[0]), lambda: path.permute_mx(),
                 lambda: path.expert_gate_up_mx(w), lambda: path.expert_down_mx(w)):
        with pytest.raises(ValueError, match="rows are bf16"):
            step()


def test_no_ffn_shape():
    with pytest.raises(ValueError, match="no expert FFN"):
        RouterDispatch(dataclasses.replace(WORKLOADS["mixtral_tiny"], ffn_dim=0, T=4), device="cpu",
                       mx=moe.MOE_MX_E2M1)


def test_inputs_that_would_go_unused_are_refused():
    """A norm in front of bf16 rows, and a residual with no norm to add it in."""
    x = torch.zeros((16, 8), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="norm"):
        path_of(None).run({"x": x, "gain": x[0], "y": None, "w": None})
    with pytest.raises(ValueError, match="residual"):
        path_of(moe.MOE_MX_E4M3).run({"x": x, "residual": x, "y": None, "w": None})
