"""The MX operators together, as RouterDispatch runs them: norm -> gate -> route ->
dispatch -> permute of MX rows -> experts on MX operands -> combine.  Each stage is
compared with its 64-bit definition on the stage before it."""
import numpy as np
import pytest
import torch

import mx_oracle as mo
import token_dispatch_moe_b200 as moe
from gpu_check import check_combine, check_dispatch, np32
from token_dispatch_moe_b200.path import RouterDispatch
from token_dispatch_moe_b200.workloads import WORKLOADS, make_inputs, make_mx_expert_weights
from test_expert_ffn_mx_gpu import check_h, f64
from test_mx_rows_gpu import assert_bits

pytestmark = pytest.mark.gpu
DEV = "cuda"
E4, E2 = moe.MOE_MX_E4M3, moe.MOE_MX_E2M1


def inputs_of(wl, norm, seed_offset=0):
    inp = make_inputs(wl, DEV, with_y=False, seed_offset=seed_offset)
    if norm:
        g = torch.Generator(device=DEV).manual_seed(17 + seed_offset)
        inp["residual"] = torch.randn((wl.T, wl.d), generator=g, device=DEV).to(torch.bfloat16)
        inp["gain"] = (1 + 0.1 * torch.randn((wl.d,), generator=g, device=DEV)).to(torch.bfloat16)
        inp["residual_out"] = torch.empty_like(inp["residual"])
    return inp


def check_path(path, wl, inp, ex, norm):
    assert path.status.item() == 0
    x = path.xn if norm else inp["x"]
    if norm:
        h, want = mo.rmsnorm(*(t.double().cpu().numpy() for t in (inp["x"], inp["residual"], inp["gain"])),
                             1e-5, lambda a: torch.from_numpy(a).float().bfloat16().double().numpy())
        assert np.array_equal(inp["residual_out"].double().cpu().numpy(), h)
        err = np.abs(path.xn.double().cpu().numpy() - want)
        assert (err <= np.abs(want) * (2.0 ** -8 + 2.0 ** -18)).all()   # as test_mx_rows_gpu
    assert_bits(path.x_mx, x.cpu())
    dest = np32(path.dest_pos)
    offsets = np32(path.offsets)
    check_dispatch(np32(path.topk_ids), np32(path.counts), offsets, np32(path.sorted_token), dest, wl.E)
    n = int(offsets[-1])
    src = torch.from_numpy(np32(path.sorted_token)[:n].astype(np.int64))
    assert torch.equal(path.xs_mx.q[:n].cpu(), path.x_mx.q.cpu()[src])
    assert torch.equal(path.xs_mx.scales[:n].cpu(), path.x_mx.scales.cpu()[src])
    oai = wl.ffn_act == "swiglu_oai"
    for e in range(wl.E):
        at = slice(int(offsets[e]), int(min(offsets[e + 1], offsets[e] + 24)))   # 24 rows of each
        if at.start == at.stop:
            continue
        b1, b3, b2 = (ex[b][e].double().cpu().numpy() if ex[b] is not None else 0.0 for b in ("b1", "b3", "b2"))
        want, bound = mo.gate_up(f64(path.xs_mx, at), f64(ex["w1"], e), f64(ex["w3"], e), b1, b3, oai, wl.d)
        check_h(path.h_mx, want, bound, at)
        want, bound = mo.down(f64(path.h_mx, at), f64(ex["w2"], e), b2, wl.ffn_dim)
        assert (np.abs(path.y[at].double().cpu().numpy() - want) <= bound).all()
    check_combine(path.out, path.y, np32(path.topk_w), dest, inp["shared"])


@pytest.mark.parametrize("name,T,mx,wmx,norm", [
    ("mixtral_tiny", 256, E4, E2, True), ("mixtral_tiny", 37, E2, E4, False),
    ("qwen3_dynk", 600, E4, E2, True), ("qwen3_dynk", 1, E4, E2, True),
    ("qwen3_dynk", 33, E4, E4, False)])
def test_chain(name, T, mx, wmx, norm):
    wl = WORKLOADS[name].scaled(T)
    inp = inputs_of(wl, norm)
    ex = make_mx_expert_weights(wl, wmx, DEV)
    path = RouterDispatch(wl, mx=mx)
    path.run(inp, experts=ex)
    torch.cuda.synchronize()
    check_path(path, wl, inp, ex, norm)


def test_chain_of_gptoss_token():
    """One token of gpt-oss: clamped SwiGLU, biases, width 2880 (padded MX rows)."""
    import dataclasses
    wl = dataclasses.replace(WORKLOADS["gptoss_top4"], T=1, E=8, skew=False)
    inp = inputs_of(wl, True)
    ex = make_mx_expert_weights(wl, E2, DEV)
    path = RouterDispatch(wl, mx=E4)
    path.run(inp, experts=ex)
    torch.cuda.synchronize()
    check_path(path, wl, inp, ex, True)


def test_chain_graphs_share_weights_and_replay():
    """Two captured graphs of two paths that share the weights, replayed in turn on two streams
    over new inputs: the bits of the eager chain."""
    wl = WORKLOADS["qwen3_dynk"].scaled(96)
    ex = make_mx_expert_weights(wl, E2, DEV)
    pairs = []
    for i in range(2):
        inp, path = inputs_of(wl, True, 100000 * i), RouterDispatch(wl, mx=E4)
        path.run(inp, experts=ex)
        torch.cuda.synchronize()
        g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        with torch.cuda.graph(g, stream=s, capture_error_mode="relaxed"):
            path.run(inp, experts=ex)
        pairs.append((inp, path, g, s))
    for turn in range(3):
        for i, (inp, path, g, s) in enumerate(pairs):
            inp["x"].copy_(inputs_of(wl, False, 1000 + 10 * turn + i)["x"])
        torch.cuda.synchronize()
        for inp, path, g, s in pairs:                    # both at once
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for inp, path, g, s in pairs:
            eager = RouterDispatch(wl, mx=E4)
            eager.run({**inp, "residual_out": torch.empty_like(inp["residual"])}, experts=ex)
            torch.cuda.synchronize()
            assert path.status.item() == 0
            n = int(eager.offsets[-1].item())
            assert torch.equal(path.topk_ids, eager.topk_ids)
            assert torch.equal(path.h_mx.q[:n], eager.h_mx.q[:n])
            assert torch.equal(path.y[:n], eager.y[:n]) and torch.equal(path.out, eager.out)


def test_padded_and_limited_blocks():
    """Blocks of moe_dispatch_limited (capacity, padding rows): the padding's rows are rows of
    the block, and the tokens' outputs are the same as without padding."""
    T, k, E, d, F = 150, 2, 8, 256, 96
    g = torch.Generator(device=DEV).manual_seed(3)
    ids = torch.randint(0, E, (T, k), generator=g, device=DEV, dtype=torch.int32)
    x = torch.randn((T, d), generator=g, device=DEV).to(torch.bfloat16)
    w = moe.MxRows.empty((E, F), d, E2)
    moe.moe_mx_quantize((torch.randn((E, F, d), generator=g, device=DEV) / 16).to(torch.bfloat16), w)
    mx = moe.MxRows.empty((T,), d, E4)
    moe.moe_mx_quantize(x, mx)
    got = []
    for pad in (1, 128):
        rows = moe.moe_dispatch_limited_rows(T, k, E, 0, pad)
        i32 = dict(dtype=torch.int32, device=DEV)
        counts, offsets = torch.empty((E,), **i32), torch.empty((E + 1,), **i32)
        st, dest = torch.empty((rows,), **i32), torch.empty((T, k), **i32)
        ws = torch.empty((max(moe.moe_dispatch_workspace_size(T, k, E), 256),), dtype=torch.uint8, device=DEV)
        moe.moe_dispatch_limited(ids, E, 0, pad, counts, offsets, st, dest, ws)
        xs = moe.MxRows(*(torch.zeros_like(t) for t in moe.MxRows.empty((rows,), d, E4)[:2]), d, E4)
        for a, b in zip(mx.as_bf16_rows(), xs.as_bf16_rows()):
            moe.moe_permute(a, dest, b)
        h = moe.MxRows.empty((rows,), F, E4)
        moe.moe_expert_gate_up_mx(xs, offsets, w, w, h)
        at = dest.long().flatten()
        got.append((h.q[at], h.scales[at]))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
