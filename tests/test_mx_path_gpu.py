"""RouterDispatch with MX activations: the chains that end before the experts' products."""
import dataclasses

import numpy as np
import pytest
import torch

import token_dispatch_moe_b200 as moe
from gpu_check import check_combine, check_dispatch, np32
from token_dispatch_moe_b200.path import RouterDispatch
from token_dispatch_moe_b200.workloads import WORKLOADS, make_inputs
from test_mx_chain_gpu import inputs_of
from test_mx_rows_gpu import assert_bits

pytestmark = pytest.mark.gpu
DEV = "cuda"
E4, E2 = moe.MOE_MX_E4M3, moe.MOE_MX_E2M1


def check_rows(path, ids):
    """The permuted MX rows are the tokens' rows."""
    offsets = np32(path.offsets)
    check_dispatch(np32(ids), np32(path.counts), offsets, np32(path.sorted_token), np32(path.dest_pos),
                   path.wl.E)
    n = int(offsets[-1])
    src = torch.from_numpy(np32(path.sorted_token)[:n].astype(np.int64))
    assert torch.equal(path.xs_mx.q[:n].cpu(), path.x_mx.q.cpu()[src])
    assert torch.equal(path.xs_mx.scales[:n].cpu(), path.x_mx.scales.cpu()[src])


@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("mx", [E4, E2])
def test_run_without_experts(mx, norm):
    """As with bf16 rows, the combine then reads the outputs that the inputs hold."""
    wl = WORKLOADS["mixtral_tiny"].scaled(61)
    inp = inputs_of(wl, norm)
    inp["y"] = make_inputs(wl, DEV)["y"]
    path = RouterDispatch(wl, mx=mx)
    out = path.run(inp)
    torch.cuda.synchronize()
    assert path.status.item() == 0 and out is path.out
    assert_bits(path.x_mx, (path.xn if norm else inp["x"]).cpu())
    check_rows(path, path.topk_ids)
    check_combine(path.out, inp["y"], np32(path.topk_w), np32(path.dest_pos), inp["shared"])


def test_run_without_experts_and_combine():
    wl = dataclasses.replace(WORKLOADS["mixtral_tiny"].scaled(33), combine=False)
    path = RouterDispatch(wl, mx=E4)
    assert path.run(inputs_of(wl, False)) is path.xs_mx
    torch.cuda.synchronize()
    check_rows(path, path.topk_ids)


def test_hash_layer():
    wl = dataclasses.replace(WORKLOADS["deepseek_v4"].scaled(50), d=256, ffn_dim=64, hash_vocab=1000)
    inp = make_inputs(wl, DEV, with_y=False)
    path = RouterDispatch(wl, mx=E4)
    assert path.run_hash_layer(inp) is path.xs_mx
    torch.cuda.synchronize()
    assert path.status.item() == 0
    assert_bits(path.x_mx, inp["x"].cpu())
    assert torch.equal(path.hash_ids, inp["tid2eid"][inp["token_ids"].long()])
    check_rows(path, path.hash_ids)
