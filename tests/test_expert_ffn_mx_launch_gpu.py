"""moe_expert_gate_up_mx and moe_expert_down_mx launched close together: a CTA pair's end, beside
kernels that take over its shared memory, and calls from several host threads."""
import threading

import pytest
import torch

import token_dispatch_moe_b200 as moe
from test_expert_ffn_mx_gpu import DEV, E2, E4, blocks, f64, filled, mx_of, randn
import mx_oracle as mo
import numpy as np

pytestmark = pytest.mark.gpu


class Call:
    """The two products over one routing: run() launches both; check() compares with the first
    run's bits, and once with the definition."""

    def __init__(self, counts, d, F, seed):
        E = len(counts)
        self.d, self.F, self.first = d, F, None
        self.off, self.offsets = blocks(counts)
        rows = int(self.off[-1])
        self.xs = mx_of(randn((rows, d), seed), E4)
        self.w1 = mx_of(randn((E, F, d), seed + 1, d ** -0.5), E2)
        self.w2 = mx_of(randn((E, d, F), seed + 2, F ** -0.5), E2)
        self.h = moe.MxRows.empty((rows,), F, E4)
        self.y = torch.empty((rows, d), dtype=torch.bfloat16, device=DEV)
        self.st = torch.zeros((1,), dtype=torch.int32, device=DEV)

    def run(self, stream=None):
        moe.moe_expert_gate_up_mx(self.xs, self.offsets, self.w1, self.w1, self.h, d_status=self.st,
                                  stream=stream)
        moe.moe_expert_down_mx(self.h, self.offsets, self.w2, self.y, d_status=self.st, stream=stream)

    def check(self):
        assert self.st.item() == 0
        got = (self.h.q.clone(), self.h.scales.clone(), self.y.clone())
        if self.first is None:
            for e in range(len(self.off) - 1):
                at = slice(int(self.off[e]), int(self.off[e + 1]))
                if at.start < at.stop:
                    want, bound = mo.down(f64(self.h, at), f64(self.w2, e), 0.0, self.F)
                    assert (np.abs(self.y[at].double().cpu().numpy() - want) <= bound).all()
            self.first = got
        for a, b in zip(got, self.first):
            assert torch.equal(a, b)
        for t in (self.h.q, self.h.scales, self.y):
            t.fill_(0)


def test_pairs_close_together():
    """Many short launches of CTA pairs, of different shapes (their barriers lie at different
    places), with single-CTA launches and the row kernels between: every launch's bits are the
    first one's."""
    calls = [Call([90, 11, 70], 256, 264, 1),        # pairs
             Call([40] * 5, 128, 72, 11),            # pairs, fewer tokens a tile
             Call([3, 8, 1], 384, 136, 21),          # one CTA a tile
             Call([700, 3, 500], 136, 392, 31)]      # pairs, several tiles a block
    for turn in range(40):
        for _ in range(5):
            for c in calls:
                c.run()
        torch.cuda.synchronize()
        for c in calls:
            c.check()


@pytest.mark.parametrize("off,status", [
    ([0, 0, 0], moe.MOE_OK), ([200, 200, 200], moe.MOE_OK), ([7, 7, 7], moe.MOE_OK),
    ([0, 150, 100], moe.MOE_ERR_DEVICE_INDEX), ([-8, 100, 200], moe.MOE_ERR_DEVICE_INDEX),
    ([0, 100, 201], moe.MOE_ERR_DEVICE_INDEX)])
def test_pairs_without_tiles(off, status):
    """Pairs that find no row, or offsets to report: they end, and write nothing."""
    E, d, F, rows = 2, 128, 72, 200
    offsets = torch.tensor(off, dtype=torch.int32, device=DEV)
    xs, w1, w2 = mx_of(randn((rows, d), 1), E4), mx_of(randn((E, F, d), 2), E2), mx_of(randn((E, d, F), 3), E2)
    h, hin = filled((rows,), F, E4), mx_of(randn((rows, F), 4), E4)
    y = torch.full((rows, d), 9.0, dtype=torch.bfloat16, device=DEV)
    for call in (lambda st: moe.moe_expert_gate_up_mx(xs, offsets, w1, w1, h, d_status=st),
                 lambda st: moe.moe_expert_down_mx(hin, offsets, w2, y, d_status=st)):
        st = torch.zeros((1,), dtype=torch.int32, device=DEV)
        call(st)
        torch.cuda.synchronize()
        assert st.item() == status
    assert (h.q == 0xA5).all() and (h.scales == 0xA5).all() and (y == 9.0).all()


@pytest.mark.parametrize("shapes", [
    [([3, 8, 1], 384, 136), ([1, 2] * 300, 64, 32), ([30, 31], 136, 72), ([12] * 64, 128, 64)],
    [([90, 11, 70], 256, 264), ([40] * 100, 128, 72), ([700, 3, 500], 136, 392), ([64] * 9, 64, 32)],
], ids=["one CTA", "pairs"])
def test_calls_of_several_host_threads(shapes):
    """Four host threads, each with its own stream, sizes and expert count (so its own shared
    memory), launch at the same time (ctypes lets the interpreter's lock go during a call): no
    call fails, and the bits are those of one thread alone."""
    calls = [Call(*s, seed=5 + 10 * i) for i, s in enumerate(shapes)]
    for c in calls:
        c.run()
    torch.cuda.synchronize()
    for c in calls:
        c.check()
    failed = launch_together([lambda s, c=c: c.run(s) for c in calls], 1500)
    assert not failed, failed[0]
    for c in calls:
        c.check()


def launch_together(steps, times):
    """step(stream) for each of steps, `times` times in a thread of its own; the errors."""
    failed, start = [], threading.Barrier(len(steps))

    def work(step):
        stream = torch.cuda.Stream()
        torch.zeros((1,), device=DEV)  # the thread's context is set up
        start.wait()
        try:
            for _ in range(times):
                step(stream)
        except moe.MoeError as e:
            failed.append(e)
        stream.synchronize()

    threads = [threading.Thread(target=work, args=(s,)) for s in steps]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    return failed
