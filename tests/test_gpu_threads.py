"""Calls of several host threads with sizes that need different amounts of shared memory: none fails another's launch,
and each gets what it gets alone. The threads make the C call itself in a loop, which runs outside of Python's lock."""
from __future__ import annotations

import ctypes
import threading

import pytest
import torch

from combine_moe_layout_gb300 import _binding as B
from gpu_common import require_gpu

pytestmark = pytest.mark.gpu


def ints(*shape):
    return torch.zeros(shape, dtype=torch.int32, device="cuda:0")


def rows(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16, device="cuda:0")


class Call:
    def __init__(self, fn, desc, *args):
        self.keep, self.err, self.stream = (desc, args), ints(1), torch.cuda.Stream()
        self.fn, self.desc = fn, ctypes.byref(desc)
        self.args = [a if a is None or isinstance(a, int) else ctypes.c_void_p(a.data_ptr()) for a in (*args, self.err)]
        self.args.append(ctypes.c_void_p(self.stream.cuda_stream))

    def __call__(self):
        return self.fn(self.desc, *self.args)


def choices(T, E):
    return torch.randint(0, E, (T, 2), generator=torch.Generator().manual_seed(E), dtype=torch.int32).cuda()


def sort(E, T=1024):
    c = Call(B.load().moe_sort, B.MoeDesc(1, T, 8, E, 2, T, B.MOE_BF16, 0), choices(T, E), rows(T, 8), None, ints(E + 1),
             rows(2 * T, 8), None, ints(T, 2))
    c.out = c.keep[1][6]
    return c


def layout(E, T=64):
    c = Call(B.load().moe_layout, B.MoeDesc(1, T, 8, E, 2, T, B.MOE_BF16, 0), choices(T, E), ints(E, 1),
             torch.zeros((E, 1), dtype=torch.int64, device="cuda:0"), ints(T, 2))
    c.out = c.keep[1][3]
    return c


def experts(E, T=16, H=128):
    g = torch.Generator().manual_seed(E)
    off = torch.arange(E + 1).mul(2 * T).div(E, rounding_mode="floor").to(torch.int32).cuda()
    x, w = (torch.randn(s, generator=g).to(torch.bfloat16).cuda() for s in ((2 * T, H), (E, H, H)))
    c = Call(B.load().moe_expert_down, B.MoeDesc(1, T, H, E, 2, T, B.MOE_BF16, 0), H, off, x, w, rows(2 * T, H))
    c.out = c.keep[1][4]
    return c


@pytest.mark.parametrize("make,sizes", [(sort, (4000, 1024)), (layout, (4096, 2600)), (experts, (600, 8))])
def test_threads_of_different_sizes(make, sizes):
    require_gpu()
    calls = [make(E) for E in sizes * 2]
    torch.cuda.synchronize()
    for c in calls:
        assert c() == B.MOE_OK
    torch.cuda.synchronize()
    want = [c.out.clone() for c in calls]
    failed = [0] * len(calls)
    start = threading.Barrier(len(calls))

    def loop(i):
        torch.cuda.set_device(0)
        start.wait()
        failed[i] = sum(calls[i]() != B.MOE_OK for _ in range(5000))

    threads = [threading.Thread(target=loop, args=(i,)) for i in range(len(calls))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert failed == [0] * len(calls)
    for c, w in zip(calls, want):
        assert B.moe_get_error(c.err, c.stream) == B.MOE_OK and torch.equal(c.out, w)
