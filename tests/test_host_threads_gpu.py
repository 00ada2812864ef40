"""The library called from host threads: a thread's first CUDA work may be one of its calls."""
import threading

import pytest
import torch

import token_dispatch_moe_b200 as moe

pytestmark = pytest.mark.gpu
DEV = "cuda"
T, d, E, F, k = 128, 128, 8, 64, 2


def in_new_thread(f):
    """f() in a host thread that has done nothing yet; its error is raised here."""
    errors = []

    def work():
        try:
            f()
        except Exception as e:  # noqa: BLE001 (raised below)
            errors.append(e)

    t = threading.Thread(target=work)
    t.start()
    t.join()
    if errors:
        raise errors[0]
    torch.cuda.synchronize()


def steps():
    """name -> (call(stream), its outputs) of every entry point that launches a kernel with an
    argument or a limit prepared on the host."""
    g = torch.Generator(device=DEV).manual_seed(1)
    rand = lambda *s: torch.randn(s, generator=g, device=DEV)
    bf = lambda *s: rand(*s).to(torch.bfloat16)
    new = lambda dt, *s: torch.zeros(s, dtype=dt, device=DEV)
    x, w, gain = bf(T, d), bf(E, d), bf(d)
    logits, ids, tw = rand(T, E), new(torch.int32, T, k), new(torch.float32, T, k)
    params = moe.RouteParams.make(E, k, moe.SCORE_SOFTMAX, 1, 1, 1, True, 1.0)
    offsets = torch.tensor([0] + [T] * E, dtype=torch.int32, device=DEV)
    w1, w2 = bf(E, F, d), bf(E, d, F)
    lg, h, y, n = new(torch.float32, T, E), new(torch.bfloat16, T, F), bf(T, d), new(torch.bfloat16, T, d)

    def mx_of(t, fmt):
        mx = moe.MxRows.empty(t.shape[:-1], t.shape[-1], fmt)
        moe.moe_mx_quantize(t, mx)
        return mx

    E4, E2 = moe.MOE_MX_E4M3, moe.MOE_MX_E2M1
    xs, w1m, w2m, h_in = mx_of(x, E4), mx_of(w1, E2), mx_of(w2, E2), mx_of(bf(T, F), E4)
    q, hm = moe.MxRows.empty((T,), d, E4), moe.MxRows.empty((T,), F, E4)
    ym, back = new(torch.bfloat16, T, d), new(torch.bfloat16, T, d)
    return {
        "gate_gemm": (lambda s: moe.moe_gate_gemm(x, w, lg, stream=s), [lg]),
        "gate_route": (lambda s: moe.moe_gate_route(x, w, None, None, params, ids, tw, stream=s), [ids, tw]),
        "route": (lambda s: moe.moe_route(logits, None, None, params, ids, tw, stream=s), [ids, tw]),
        "expert_gate_up": (lambda s: moe.moe_expert_gate_up(x, offsets, w1, w1, h, stream=s), [h]),
        "expert_down": (lambda s: moe.moe_expert_down(h, offsets, w2, y, stream=s), [y]),
        "add_rmsnorm": (lambda s: moe.moe_add_rmsnorm(x, None, gain, 1e-5, y=n, stream=s), [n]),
        "mx_quantize": (lambda s: moe.moe_mx_quantize(x, q, s), [q.q, q.scales]),
        "mx_dequantize": (lambda s: moe.moe_mx_dequantize(xs, back, s), [back]),
        "expert_gate_up_mx": (lambda s: moe.moe_expert_gate_up_mx(xs, offsets, w1m, w1m, hm, stream=s),
                              [hm.q, hm.scales]),
        "expert_down_mx": (lambda s: moe.moe_expert_down_mx(h_in, offsets, w2m, ym, stream=s), [ym]),
    }


NAMES = ["gate_gemm", "gate_route", "route", "expert_gate_up", "expert_down", "add_rmsnorm",
         "mx_quantize", "mx_dequantize", "expert_gate_up_mx", "expert_down_mx"]


@pytest.mark.parametrize("own_stream", [True, False])
@pytest.mark.parametrize("name", NAMES)
def test_first_call_of_a_thread(name, own_stream):
    call, outs = steps()[name]
    stream = torch.cuda.Stream() if own_stream else None
    torch.cuda.synchronize()
    call(stream)
    torch.cuda.synchronize()
    want = [t.clone() for t in outs]
    for t in outs:
        t.zero_()
    torch.cuda.synchronize()
    in_new_thread(lambda: call(stream))
    for a, b in zip(outs, want):
        assert torch.equal(a, b)


def sized(kind, i):
    """(call(stream), outputs) of one entry point at its i-th size: the sizes ask for different
    amounts of shared memory."""
    g = torch.Generator(device=DEV).manual_seed(10 + i)
    rand = lambda *s: torch.randn(s, generator=g, device=DEV)
    bf = lambda *s: rand(*s).to(torch.bfloat16)
    n = (8, 64, 200, 512)[i]
    if kind == "gate_gemm":
        x, w, out = bf(300, 256), bf(n, 256), torch.zeros((300, n), device=DEV)
        return lambda s: moe.moe_gate_gemm(x, w, out, stream=s), [out]
    if kind in ("expert_gate_up", "expert_down"):
        N, rows = (16, 96, 128, 160)[i], 256
        offsets = torch.tensor([0] * (n // 2) + [rows] * (n // 2 + 1), dtype=torch.int32, device=DEV)
        if kind == "expert_gate_up":
            x, w, out = bf(rows, 64), bf(n, N, 64), torch.zeros((rows, N), dtype=torch.bfloat16, device=DEV)
            return lambda s: moe.moe_expert_gate_up(x, offsets, w, w, out, stream=s), [out]
        x, w, out = bf(rows, 64), bf(n, N, 64), torch.zeros((rows, N), dtype=torch.bfloat16, device=DEV)
        return lambda s: moe.moe_expert_down(x, offsets, w, out, stream=s), [out]
    k_max = 4 if kind == "route" else 12
    E_ = (32, 64, 256, 512)[i] if kind == "route" else (36, 128, 260, 512)[i]
    T_ = (50, 3000, 700, 9000)[i]
    logits, ids = rand(T_, E_), torch.zeros((T_, k_max), dtype=torch.int32, device=DEV)
    tw = torch.zeros((T_, k_max), device=DEV)
    params = moe.RouteParams.make(E_, k_max, moe.SCORE_SOFTMAX, 1, 1, 1, True, 1.0)
    return lambda s: moe.moe_route(logits, None, None, params, ids, tw, stream=s), [ids, tw]


class Recorder:
    """The library's handle, keeping the last call: (function, arguments)."""

    def __init__(self, lib):
        self.lib, self.last = lib, None

    def __getattr__(self, name):
        fn = getattr(self.lib, name)

        def call(*args):
            self.last = fn, args
            return fn(*args)

        return call


@pytest.mark.parametrize("kind", ["gate_gemm", "expert_gate_up", "expert_down", "route", "route_k12"])
def test_sizes_of_several_threads_at_once(kind, monkeypatch):
    """Four host threads launch one entry point at sizes of different shared memory, with nothing
    but the C call in their loops: no call fails, and the bits are those of one thread alone."""
    recorder = Recorder(moe.load_library())
    monkeypatch.setattr(moe, "_lib", recorder)
    jobs = []
    for i in range(4):
        call, outs = sized(kind, i)
        stream = torch.cuda.Stream()
        torch.cuda.synchronize()
        call(stream)
        torch.cuda.synchronize()
        jobs.append((*recorder.last, outs, [t.clone() for t in outs], stream, call))  # call: the inputs
    failed, start = [], threading.Barrier(4)

    def work(fn, args):
        torch.zeros((1,), device=DEV)
        start.wait()
        failed.extend(s for s in (fn(*args) for _ in range(20000)) if s != moe.MOE_OK)

    threads = [threading.Thread(target=work, args=job[:2]) for job in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed, failed[:5]
    for _, _, outs, want, *_ in jobs:
        for a, b in zip(outs, want):
            assert torch.equal(a, b)
