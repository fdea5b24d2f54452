"""The router (moe_gate, moe_gate_grad) against numpy in 64 bits.

Choices have to be equal. Where they are made on logits (no bias, no group sums)
any input will do; where a 32-bit score decides, the test first checks that its
inputs keep the scores 1e-5 apart, far more than 32-bit rounding.

Bars. u = 2^-24. A weight is a quotient of exponentials: expf and the division
are within 4 u, its argument l - max is off by at most 32 u for the |l - max| <= 32
here, and a sum of 1024 terms as 32 in a row per lane and 5 across takes 37
roundings: W = 128 u relative covers them twice. A gradient element is a product
of such scores with (g - mean), whose terms cancel: 4 W times the sum of the
magnitudes, plus one bf16 rounding (2^-8 of the element) for bf16 logits."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from combine_moe_layout_gb300 import _binding as B
from gpu_common import Guarded, require_gpu

pytestmark = pytest.mark.gpu
W = 128 * 2.0 ** -24


def desc(n, E, k):
    return B.MoeDesc(1, n, 8, E, k, max(n, 1), B.MOE_BF16, 0)


def opts(score="softmax", renorm=False, groups=0, keep=0, top=0, bf16=False, scale=1.0):
    return B.MoeGateOpts(B.MOE_SCORE_SOFTMAX if score == "softmax" else B.MOE_SCORE_SIGMOID, int(renorm), groups,
                         keep, top, int(bf16), scale)


def scores(l, score):
    l = np.minimum(l, np.finfo(np.float32).max)
    if score == "sigmoid":
        return 1.0 / (1.0 + np.exp(-l))
    m = l.max(axis=1, keepdims=True)
    m = np.where(np.isfinite(m), m, 0.0)
    p = np.exp(l - m)
    s = p.sum(axis=1, keepdims=True)
    return p / np.where(s > 0, s, 1.0)


def plain_gate(l, o, k, bias=None, check_margin=None):
    """ids and weights, one token and one choice at a time."""
    n, E = l.shape
    score = "softmax" if o.score == B.MOE_SCORE_SOFTMAX else "sigmoid"
    s = scores(l, score)
    ids = np.full((n, k), -1, dtype=np.int64)
    for t in range(n):
        sel = l[t].copy() if bias is None else s[t] + bias
        avail = l[t] > -np.inf
        if bias is not None:
            avail &= sel > -np.inf
        if o.num_groups > 1:
            size = E // o.num_groups
            gv = l[t] if bias is None and o.group_top == 1 else s[t] + (0 if bias is None else bias)
            gs = []
            for g in range(o.num_groups):
                v = sorted((gv[e] for e in range(g * size, (g + 1) * size) if avail[e]), reverse=True)
                gs.append(sum(v[:o.group_top]) if v else -np.inf)
            order = sorted(range(o.num_groups), key=lambda g: (-gs[g], g))
            if check_margin and o.keep_groups < o.num_groups and np.isfinite(gs[order[o.keep_groups]]):
                assert abs(gs[order[o.keep_groups - 1]] - gs[order[o.keep_groups]]) > check_margin
            kept = {g for g in order[:o.keep_groups] if gs[g] > -np.inf}
            avail &= np.array([e // size in kept for e in range(E)])
        cand = [e for e in sorted(range(E), key=lambda e: (-sel[e], e)) if avail[e]]
        if check_margin and bias is not None:
            v = [sel[e] for e in cand[:k + 1]]
            assert all(a - b > check_margin for a, b in zip(v, v[1:]))
        ids[t, :len(cand[:k])] = cand[:k]
    return ids, plain_weights(l, ids, score, o.renormalize, o.scale)


def plain_weights(l, ids, score, renorm, scale):
    s = np.take_along_axis(scores(l, score), np.maximum(ids, 0), axis=1) * (ids >= 0)
    if renorm:
        tot = s.sum(axis=1, keepdims=True)
        s = np.where(tot > 0, s / np.where(tot > 0, tot, 1.0), 0.0)
    return s * scale


def plain_grad(l, ids, g, score, renorm, scale):
    """dL/dl, and the sum of magnitudes its rounding bar is taken from."""
    n, E = l.shape
    live = ids >= 0
    at = np.maximum(ids, 0)
    s = scores(l, score)
    c = np.take_along_axis(s, at, axis=1) * live
    g = g * live * scale
    if renorm:
        tot = c.sum(axis=1, keepdims=True)
        safe = np.where(tot > 0, tot, 1.0)
        ds = (g - (g * c).sum(axis=1, keepdims=True) / safe) / safe * (tot > 0)
        mag = (np.abs(g) + (np.abs(g) * c).sum(axis=1, keepdims=True) / safe) / safe
    else:
        ds, mag = g, np.abs(g)
    d, bar = np.zeros((n, E)), np.zeros((n, E))
    rows = np.arange(n)[:, None]
    if score == "sigmoid":
        np.add.at(d, (rows, at), ds * c * (1 - c) * live)
        np.add.at(bar, (rows, at), mag * c * live)
    else:
        np.add.at(d, (rows, at), ds * c * live)
        np.add.at(bar, (rows, at), mag * c * live)
        if not renorm:
            d -= s * (ds * c).sum(axis=1, keepdims=True)
            bar += s * (mag * c).sum(axis=1, keepdims=True)
    return d, bar


def run_gate(l, o, k, bias=None):
    n, E = l.shape
    idx, w = Guarded((n, k), torch.int32, "cuda:0"), Guarded((n, k), torch.float32, "cuda:0")
    err = torch.zeros(1, dtype=torch.int32, device="cuda:0")
    B.moe_gate(desc(n, E, k), o, l, bias, idx.t, w.t, err)
    status = B.moe_get_error(err)
    assert idx.guards_intact() and w.guards_intact()
    return idx.t, w.t, status


def run_grad(l, o, idx, g):
    n, E = l.shape
    out = Guarded((n, E), l.dtype, "cuda:0")
    err = torch.zeros(1, dtype=torch.int32, device="cuda:0")
    B.moe_gate_grad(desc(n, E, idx.shape[1]), o, l, idx, g, out.t, err)
    status = B.moe_get_error(err)
    assert out.guards_intact()
    return out.t, status


def logits(n, E, bf16, seed=0, spread=2.0):
    g = torch.Generator().manual_seed(seed)
    l = torch.randn((n, E), generator=g) * spread
    return (l.to(torch.bfloat16) if bf16 else l).cuda()


def check(l, o, k, bias=None, margin=None):
    idx, w, status = run_gate(l, o, k, bias)
    assert status == B.MOE_OK
    l64 = l.double().cpu().numpy()
    b64 = None if bias is None else bias.double().cpu().numpy()
    ids, wr = plain_gate(l64, o, k, b64, margin)
    assert np.array_equal(idx.cpu().numpy(), ids)
    got = w.double().cpu().numpy()
    assert (np.abs(got - wr) <= W * np.abs(wr) + 2.0 ** -140).all()
    g = torch.randn(idx.shape, generator=torch.Generator().manual_seed(3)).cuda()
    d, status = run_grad(l, o, idx, g)
    assert status == B.MOE_OK
    score = "softmax" if o.score == B.MOE_SCORE_SOFTMAX else "sigmoid"
    want, bar = plain_grad(l64, ids, g.double().cpu().numpy(), score, o.renormalize, o.scale)
    tol = 4 * W * bar + (2.0 ** -8 * np.abs(want) if l.dtype == torch.bfloat16 else 0.0) + 2.0 ** -120
    assert (np.abs(d.double().cpu().numpy() - want) <= tol).all()


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("n,E,k", [(1, 256, 8), (37, 8, 2), (5, 1, 1), (19, 7, 3), (64, 60, 6), (9, 130, 16),
                                   (33, 257, 5), (3, 1024, 8), (7, 16, 16)])
def test_gate_and_gradient(n, E, k, score, renorm, bf16):
    require_gpu()
    check(logits(n, E, bf16, seed=n + E), opts(score, renorm, bf16=bf16, scale=2.5), k)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups,keep,top,k", [(256, 8, 4, 2, 8), (160, 8, 3, 1, 6), (96, 3, 2, 3, 8), (32, 32, 9, 1, 8),
                                                 (1023, 3, 1, 5, 8), (60, 5, 5, 12, 4), (68, 17, 4, 2, 16)])
def test_groups(E, groups, keep, top, k, score):
    require_gpu()
    check(logits(23, E, False, seed=E, spread=1.0), opts(score, True, groups, keep, top), k, margin=1e-6)


def test_single_member_groups_follow_the_logits_under_ties():
    """bf16 logits on a coarse grid: equal group scores and equal logits go to the lowest index."""
    require_gpu()
    l = (logits(200, 64, True, seed=9) * 2).round().to(torch.bfloat16)
    for o in (opts("sigmoid", True, 8, 3, 1, True), opts("softmax", False, bf16=True)):
        check(l, o, 8)


def test_close_and_saturated_logits_keep_their_order():
    """Scores that round to one 32-bit value are still told apart by the logits."""
    require_gpu()
    l = torch.arange(64, dtype=torch.float32).mul_(0.25).add_(20.0).flip(0)[None].repeat(3, 1)
    l = l[:, torch.randperm(64, generator=torch.Generator().manual_seed(1))].contiguous().cuda()
    check(l, opts("sigmoid"), 8)
    far = torch.full((2, 40), -300.0)
    far[:, 5] = 300.0
    far[:, 7:12] = torch.arange(5) - 200.0
    idx, w, status = run_gate(far.cuda(), opts("softmax"), 4)
    assert status == B.MOE_OK and idx[0].tolist() == [5, 11, 10, 9] and w[0].tolist() == [1.0, 0.0, 0.0, 0.0]


def test_values_that_differ_in_their_last_bits_only():
    """fp32 logits that agree in all but the lowest few bits, among the chosen, across the k-th place and below it, and
    many equal ones: the order is still the logits', ties to the lowest expert."""
    require_gpu()
    for E in (40, 256, 700, 1024):
        g = torch.Generator().manual_seed(E)
        l = torch.randn((60, E), generator=g)
        base = torch.tensor([3.0, -0.5])[torch.arange(60) % 2]
        near = (base[:, None].view(-1, 1).expand(60, 12).contiguous().view(torch.int32)
                + torch.randint(0, 6, (60, 12), generator=g, dtype=torch.int32)).view(torch.float32)
        at = torch.argsort(torch.rand((60, E), generator=g), 1)[:, :12]
        l.scatter_(1, at, near)
        l[::2] = torch.where(torch.rand((30, E), generator=g) < 0.3, l[::2], torch.full_like(l[::2], -4.0))
        for k in (1, 5, 16):
            check(l.cuda(), opts("sigmoid", True), k)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("E", [100, 256, 1024])
def test_the_chosen_are_neighbours(E, dtype):
    """The largest logits lie next to one another and a fixed distance apart, so that one lane holds many of them."""
    require_gpu()
    g = torch.Generator().manual_seed(E)
    l = torch.rand((5, E), generator=g).sub_(9).to(dtype)
    high = torch.arange(16) / 8 + 1
    l[0, 4:20] = high.to(dtype)
    l[1, torch.arange(16) // 4 * (E // 4 // 4 * 4) + torch.arange(16) % 4] = high.to(dtype)
    l[2, torch.arange(4) + 8] = high[:4].to(dtype)
    l[3, :] = float("-inf")
    l[3, 8:13] = high[:5].to(dtype)
    l[4, [8, 9, 10, 11, E - 1]] = high[:5].to(dtype)
    for k in (1, 4, 5, 8, 16):
        check(l.cuda(), opts("sigmoid", True, bf16=dtype == torch.bfloat16), k)


@pytest.mark.parametrize("groups", [0, 4])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_bias_selects_and_does_not_weigh(score, groups):
    require_gpu()
    E, n, k = 64, 17, 6
    g = torch.Generator().manual_seed(5)
    step = 0.9 / E
    s = torch.stack([torch.randperm(E, generator=g) for _ in range(n)]).double().add_(0.5).mul_(step)
    if score == "sigmoid":
        l = torch.log(s / (1 - s))
    else:
        l = torch.log(s / s.sum(1, keepdim=True))
        step = float(step / s.sum(1)[0])
    bias = (torch.randint(0, 4, (E,), generator=g).double() * 0.37 * step).float().cuda()
    o = opts(score, True, groups, 2 if groups else 0, 3 if groups else 0)
    check(l.float().cuda(), o, k, bias, margin=1e-5)


@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_unavailable_experts(score, renorm):
    """-inf logits are never chosen; rows with fewer than k left, with one left, and with none."""
    require_gpu()
    l = logits(6, 40, False, seed=2)
    l[0, :] = -float("inf")
    l[1, 1:] = -float("inf")
    l[2, 3:] = -float("inf")
    l[3, ::2] = -float("inf")
    l[4, 7] = float("inf")
    l[5, :] = -float("inf")
    l[5, 39] = torch.finfo(torch.float32).min
    check(l, opts(score, renorm), 5)
    idx, w, _ = run_gate(l, opts(score, renorm), 5)
    assert idx[0].tolist() == [-1] * 5 and w[0].tolist() == [0.0] * 5
    assert idx[1].tolist() == [0, -1, -1, -1, -1] and int(idx[4, 0]) == 7
    g = torch.ones(idx.shape, device="cuda:0")
    d, _ = run_grad(l, opts(score, renorm), idx, g)
    assert bool(torch.isfinite(d).all()) and bool((d[0] == 0).all())


def test_groups_with_nothing_available():
    require_gpu()
    l = logits(4, 64, False, seed=4)
    l[0, 16:] = -float("inf")   # one group left
    l[1, :] = -float("inf")     # none
    l[2, 1:63] = -float("inf")  # one expert in the first and one in the last
    check(l, opts("sigmoid", True, 4, 2, 2), 8)


def test_very_negative_sigmoid_logits_give_zero_weights():
    require_gpu()
    l = torch.full((2, 16), -200.0, device="cuda:0")
    for renorm in (False, True):
        idx, w, status = run_gate(l, opts("sigmoid", renorm), 4)
        assert status == B.MOE_OK and idx.tolist() == [[0, 1, 2, 3]] * 2
        d, _ = run_grad(l, opts("sigmoid", renorm), idx, torch.ones((2, 4), device="cuda:0"))
        assert bool((w == 0).all()) and bool((d == 0).all())


def test_nan_logits_are_reported_and_left_out():
    require_gpu()
    l = logits(3, 16, False, seed=6)
    l[1, 4] = float("nan")
    idx, w, status = run_gate(l, opts("softmax", True), 16)  # every expert is asked for
    assert status == B.MOE_EINVAL
    assert 4 not in idx[1].tolist() and int(idx[1, 15]) == -1 and bool(torch.isfinite(w).all())
    bias = torch.zeros(32, device="cuda:0")
    bias[9] = float("nan")
    idx, _, status = run_gate(logits(3, 32, False, seed=6), opts("sigmoid"), 8, bias)
    assert status == B.MOE_EINVAL and bool((idx != 9).all())


def test_gradient_reports_an_invalid_id_and_adds_up_a_repeated_one():
    require_gpu()
    l = logits(2, 12, False, seed=8)
    idx = torch.tensor([[3, 12, -1], [5, 5, 0]], dtype=torch.int32, device="cuda:0")
    g = torch.tensor([[1.0, 9.0, 9.0], [0.5, 0.25, 1.0]], device="cuda:0")
    d, status = run_grad(l, opts("sigmoid"), idx, g)
    assert status == B.MOE_EINVAL
    s = scores(l.double().cpu().numpy(), "sigmoid")
    want = np.zeros((2, 12))
    want[0, 3] = s[0, 3] * (1 - s[0, 3])
    want[1, 5] = 0.75 * s[1, 5] * (1 - s[1, 5])
    want[1, 0] = s[1, 0] * (1 - s[1, 0])
    assert (np.abs(d.double().cpu().numpy() - want) <= 8 * W * np.abs(want)).all()


@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_gradient_against_differences(score, renorm):
    """Central differences of the weights' formula in 64 bits, h = 1e-5: their own error is about h^2 + 2^-52 / h,
    below 1e-9."""
    require_gpu()
    n, E, k, h = 3, 20, 4, 1e-5
    l = logits(n, E, False, seed=11, spread=1.0)
    o = opts(score, renorm, scale=1.5)
    idx, _, _ = run_gate(l, o, k)
    g = torch.randn((n, k), generator=torch.Generator().manual_seed(12)).cuda()
    d, _ = run_grad(l, o, idx, g)
    l64, g64, ids = l.double().cpu().numpy(), g.double().cpu().numpy(), idx.cpu().numpy().astype(np.int64)
    _, bar = plain_grad(l64, ids, g64, score, renorm, 1.5)
    for e in range(E):
        lo, hi = l64.copy(), l64.copy()
        lo[:, e] -= h
        hi[:, e] += h
        diff = ((plain_weights(hi, ids, score, renorm, 1.5) - plain_weights(lo, ids, score, renorm, 1.5)) * g64).sum(1)
        assert (np.abs(d[:, e].double().cpu().numpy() - diff / (2 * h)) <= 4 * W * bar[:, e] + 1e-8).all()


def test_unaligned_rows_and_another_stream():
    """A base that is only element-aligned takes the scalar loads; the call runs on the stream it is given."""
    require_gpu()
    n, E, k = 50, 64, 4
    whole = torch.zeros(n * E + 1, device="cuda:0")
    l = whole[1:].view(n, E)
    l.copy_(logits(n, E, False, seed=14))
    check(l, opts("softmax", True), k)
    s = torch.cuda.Stream()
    idx = torch.empty((n, k), dtype=torch.int32, device="cuda:0")
    w = torch.empty((n, k), device="cuda:0")
    err = torch.zeros(1, dtype=torch.int32, device="cuda:0")
    torch.cuda.synchronize()
    B.moe_gate(desc(n, E, k), opts("softmax", True), l, None, idx, w, err, stream=s)
    s.synchronize()
    i2, w2, _ = run_gate(l, opts("softmax", True), k)
    assert torch.equal(idx, i2) and torch.equal(w, w2)


def test_no_tokens():
    require_gpu()
    err = torch.zeros(1, dtype=torch.int32, device="cuda:0")
    none = torch.empty((0, 8), device="cuda:0")
    i = torch.empty((0, 2), dtype=torch.int32, device="cuda:0")
    w = torch.empty((0, 2), device="cuda:0")
    B.moe_gate(desc(0, 8, 2), opts(), none, None, i, w, err)
    B.moe_gate_grad(desc(0, 8, 2), opts(), none, i, w, none, err)
    assert B.moe_get_error(err) == B.MOE_OK
