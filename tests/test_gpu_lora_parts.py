"""moe_lora_linear with u in two parts, against its formula in 64 bits.

Bar of y as for one part (test_gpu_lora.py) but for u's own rounding: what rounding left, at most 2^-9 of u, is rounded
to bf16 once more, which leaves 2^-18 |u| (taken as 2^-16), after (K + 2) 2^-22 s sum |x a| of its sum in fp32; and the
adapter's products are 2 rank."""
from __future__ import annotations

import ctypes

import pytest
import torch

from combine_moe_layout_gb300 import _binding as B
from gpu_common import Guarded, require_gpu
from test_gpu_lora import A22, bf16, ids_of

pytestmark = pytest.mark.gpu


def run(x, w, la, lb, sc, ids, parts=2, num_sms=0):
    T, K = x.shape
    A, r = la.shape[0], la.shape[1]
    d = B.MoeLoraDesc(T, K, w.shape[0], r, A, num_sms, parts)
    y = Guarded((T, w.shape[0]), torch.bfloat16, "cuda:0")
    u = Guarded((max(parts, 1), T, r), torch.bfloat16, "cuda:0")
    err = torch.zeros(1, dtype=torch.int32, device="cuda:0")
    B.moe_lora_linear(d, x, w, la, lb, sc, ids, u.t, y.t, err)
    status = B.moe_get_error(err)
    assert y.guards_intact() and u.guards_intact()
    return y.t, status


def reference(x, w, la, lb, sc, ids):
    x, w = x.double(), w.double()
    K = x.shape[1]
    y, bar = x @ w.t(), (K + 2) * A22 * (x.abs() @ w.abs().t())
    for a in range(la.shape[0]):
        t = (ids == a).nonzero().view(-1)
        if not t.numel():
            continue
        s = float(sc[a]) if sc is not None else 1.0
        aa, bb = la[a].double(), lb[a].double()
        u = s * (x[t] @ aa.t())
        du = 2.0 ** -16 * u.abs() + (K + 2) * A22 * abs(s) * (x[t].abs() @ aa.abs().t())
        y[t] += u @ bb.t()
        bar[t] += du @ bb.abs().t() + (2 * aa.shape[0] + 2) * A22 * ((u.abs() + du) @ bb.abs().t())
    return y, bar + 2.0 ** -8 * y.abs()


def operands(T, K, N, r, A, mix, seed=0):
    la, lb = bf16((A, r, K), seed + 2, K ** -0.5), bf16((A, N, r), seed + 3, r ** -0.5)
    sc = torch.rand(A, generator=torch.Generator().manual_seed(seed + 4)).add(0.25).cuda()
    return bf16((T, K), seed), bf16((N, K), seed + 1, K ** -0.5), la, lb, sc, ids_of(T, A, mix, seed)


SHAPES = [(1, 4096, 4096, 16, 8, "one"), (1, 72, 136, 256, 3, "one"), (2, 8, 8, 8, 3, "tokens"), (31, 1000, 264, 64, 40, "tokens"),
          (64, 7168, 2048, 16, 32, "tokens"), (65, 200, 520, 40, 5, "runs"), (127, 640, 384, 128, 7, "tokens"),
          (128, 512, 256, 256, 4, "tokens"), (300, 328, 1032, 72, 9, "runs"), (389, 2056, 4104, 24, 12, "tokens"),
          (260, 1032, 72, 136, 30, "tokens"), (1000, 64, 128, 8, 1000, "tokens"), (2048, 512, 5128, 64, 16, "runs"),
          (1500, 264, 8192, 16, 128, "tokens"), (4096, 192, 2048, 200, 3, "runs"), (700, 64, 16384, 8, 2, "none")]


@pytest.mark.parametrize("T,K,N,r,A,mix", SHAPES)
def test_against_the_formula(T, K, N, r, A, mix):
    require_gpu()
    ops = operands(T, K, N, r, A, mix)
    y, status = run(*ops)
    want, bar = reference(*ops)
    assert status == B.MOE_OK and bool(((y.double() - want).abs() <= bar).all())
    assert torch.equal(run(*ops)[0], y)


@pytest.mark.parametrize("T,K,N,r,A", [(1, 512, 264, 16, 3), (50, 512, 264, 32, 4), (200, 512, 520, 64, 4)])
def test_an_adapter_that_cancels(T, K, N, r, A):
    """y = u_0 b - u_1 b with u_0 and u_1 nearly alike and no base projection: what is left is 2^-9 of either, and one
    part's rounding would be as large as y. Bars as above (y's own rounding goes by y)."""
    require_gpu()
    x, w, la, lb, sc, ids = operands(T, K, N, r, A, "tokens", 7)
    w.zero_()
    ids.clamp_(min=0)
    la[:, 1] = la[:, 0]
    la[:, 1, :8] = la[:, 0, :8] * 0.75
    lb.zero_()
    lb[:, :, 0] = 1.0
    lb[:, :, 1] = -1.0
    y, status = run(x, w, la, lb, sc, ids)
    want, bar = reference(x, w, la, lb, sc, ids)
    assert status == B.MOE_OK and bool(((y.double() - want).abs() <= bar).all())


def test_zero_and_one_part_are_the_same():
    require_gpu()
    for T, mix in ((1, "one"), (40, "tokens"), (700, "runs")):
        ops = operands(T, 264, 520, 24, 3, mix)
        assert torch.equal(run(*ops, parts=0)[0], run(*ops, parts=1)[0])


def test_rows_that_are_not_finite_and_adapters_out_of_use():
    """Infinities and NaN of a row stay in it; an infinite u has no second part, so its row is what one part gives."""
    require_gpu()
    x, w, la, lb, _, _ = operands(150, 256, 264, 16, 4, "tokens")
    ids = ids_of(150, 3, "tokens", 5)
    clean, _ = run(x, w, la, lb, None, ids)
    la[3], lb[3] = float("nan"), float("inf")
    x[7], x[140] = float("nan"), float("inf")
    ids[140] = 0
    y, status = run(x, w, la, lb, None, ids)
    one, _ = run(x, w, la, lb, None, ids, parts=1)
    keep = torch.ones(150, dtype=torch.bool, device="cuda:0")
    keep[7] = keep[140] = False
    assert status == B.MOE_OK and torch.equal(y[keep], clean[keep])
    assert bool(torch.isnan(y[7]).all()) and torch.equal(torch.isnan(y[140]), torch.isnan(one[140]))


def test_refusals():
    require_gpu()
    p = [ctypes.c_void_p(1 << 20)] * 9
    for parts, T in ((3, 4), (-1, 4), (2, 1 << 30)):
        d = B.MoeLoraDesc(T, 64, 64, 16, 2, 0, parts)
        assert B.load().moe_lora_linear(ctypes.byref(d), *p, None) == B.MOE_EINVAL  # before any address is used
