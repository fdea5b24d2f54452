"""moe_gate_grad where a score is close to one: the factor 1 - s and the difference from the weighted mean are small
next to what they are made of, and still have to be right to their own size.

With c = scale g, s the chosen scores, v the renormalised ones, S their sum and t the largest chosen entry:

  sigmoid               dl_j = c_j s_j (1 - s_j),                   1 - s_j = 1 / (1 + exp(l_j))
  sigmoid, renormalised dl_j = m_j / S s_j (1 - s_j),
  softmax, renormalised dl_j = v_j m_j,                             m_j = sum_i v_i (c_j - c_i)
  softmax               dl_e = s_e (c_e [e chosen] - sum_j c_j s_j) = s_e sum_i s_i (c_e - c_i) over all experts

A sum of products of differences is good to its own terms when the largest score meets only differences: the bar is
W = 128 * 2^-24 of sum_i s_i |c_j - c_i| with the terms of i != t taken as s_i (|c_j| + |c_i|). W is the bar that the
weights have: exponentials and quotients within 4 units of 2^-24, arguments off by at most 32, sums of 37 roundings,
all taken twice. Three such factors meet in one element: 4 W."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from combine_moe_layout_gb300 import _binding as B
from gpu_common import require_gpu

pytestmark = pytest.mark.gpu
W = 128 * 2.0 ** -24


def run(l, ids, g, score, renorm, scale):
    n, E = l.shape
    d = torch.empty_like(l)
    err = torch.zeros(1, dtype=torch.int32, device="cuda:0")
    o = B.MoeGateOpts(B.MOE_SCORE_SOFTMAX if score == "softmax" else B.MOE_SCORE_SIGMOID, int(renorm), 0, 0, 0, 0, scale)
    B.moe_gate_grad(B.MoeDesc(1, n, 8, E, ids.shape[1], n, B.MOE_BF16, 0), o, l, ids, g, d, err)
    assert B.moe_get_error(err) == B.MOE_OK
    return d.double().cpu().numpy()


def mean_differences(p, c):
    """sum_i p_i (c_j - c_i) for every j, and its bar, with the largest p apart."""
    t = p.argmax()
    rest = np.arange(len(p)) != t
    diff = c[:, None] - c[None, :]
    m = (p[None, :] * diff).sum(1)
    mag = p[t] * np.abs(c - c[t]) + (p[None, rest] * (np.abs(c)[:, None] + np.abs(c)[None, rest])).sum(1)
    return m, mag


def formula(l, ids, g, score, renorm, scale):
    n, E = l.shape
    want, bar = np.zeros((n, E)), np.zeros((n, E))
    for t in range(n):
        at = ids[t]
        c = scale * g[t]
        if score == "sigmoid":
            s, q = 1 / (1 + np.exp(-l[t, at])), 1 / (1 + np.exp(l[t, at]))
            if renorm:
                m, mag = mean_differences(s / s.sum(), c)
                want[t, at], bar[t, at] = m / s.sum() * s * q, mag / s.sum() * s * q
            else:
                want[t, at], bar[t, at] = c * s * q, np.abs(c) * s * q
        elif renorm:
            p = np.exp(l[t, at] - l[t, at].max())
            p /= p.sum()
            m, mag = mean_differences(p, c)
            want[t, at], bar[t, at] = p * m, p * mag
        else:
            p = np.exp(l[t] - l[t].max())
            p /= p.sum()
            full = np.zeros(E)
            full[at] = c
            m, mag = mean_differences(p, full)
            want[t], bar[t] = p * m, p * mag
    return want, bar


def check(l, ids, g, score, renorm, scale=1.5):
    require_gpu()
    got = run(l.cuda(), ids.cuda(), g.cuda(), score, renorm, scale)
    want, bar = formula(l.double().numpy(), ids.numpy().astype(np.int64), g.double().numpy(), score, renorm, scale)
    assert (np.abs(got - want) <= 4 * W * bar + 2.0 ** -120).all()


def inputs(E, k, low, high, seed):
    """Rows whose chosen logits go from `low` to `high` above the others."""
    gen = torch.Generator().manual_seed(seed)
    n = 33
    l = torch.rand((n, E), generator=gen) * 2 - 1
    ids = torch.argsort(torch.rand((n, E), generator=gen), 1)[:, :k].to(torch.int32)
    up = torch.linspace(low, high, n)[:, None] - torch.rand((n, k), generator=gen) * 3
    l.scatter_(1, ids.long(), up)
    return l, ids, torch.randn((n, k), generator=gen)


@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("E,k", [(8, 1), (64, 4), (256, 8)])
def test_sigmoid_of_large_logits(E, k, renorm):
    check(*inputs(E, k, 8.0, 40.0, E + k), "sigmoid", renorm)


@pytest.mark.parametrize("E,k", [(8, 1), (12, 2), (64, 4), (256, 8), (1024, 3)])
def test_softmax_of_one_large_logit(E, k):
    """One choice far above all others: its gradient is what the others leave."""
    l, ids, g = inputs(E, k, 0.0, 0.5, E)
    l[torch.arange(33), ids[:, k // 2].long()] = torch.linspace(4.0, 40.0, 33)
    check(l, ids, g, "softmax", False)
    check(l, ids, g, "softmax", True)
    check(l, ids, g, "sigmoid", True)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_equal_gradients_and_equal_logits(score):
    """Gradients that are all alike leave only rounding for the renormalised weights, and for two equal largest logits
    one of them counts as the largest."""
    l, ids, g = inputs(64, 4, 3.0, 20.0, 1)
    check(l, ids, torch.full_like(g, 0.7), score, True)
    l[:, :] = l.round()
    l[torch.arange(33), ids[:, 0].long()] = l[torch.arange(33), ids[:, 1].long()] = 9.0
    for renorm in (False, True):
        check(l, ids, g, score, renorm)


def test_the_largest_logit_is_not_among_the_chosen():
    """A caller's own ids: the row's largest score has no gradient of its own."""
    l, ids, g = inputs(64, 4, 1.0, 2.0, 2)
    for t in range(33):
        free = next(e for e in range(64) if e not in ids[t].tolist())
        l[t, free] = 2.0 + t
    check(l, ids, g, "softmax", False)


@pytest.mark.parametrize("score,renorm", [("softmax", False), ("softmax", True), ("sigmoid", False), ("sigmoid", True)])
def test_an_expert_named_twice(score, renorm):
    """Its entries are two choices of equal score whose terms add up (the formulas per entry, added where they meet)."""
    require_gpu()
    l = torch.randn((5, 12), generator=torch.Generator().manual_seed(4))
    ids = torch.tensor([[5, 5, 0], [1, 2, 1], [3, 3, 3], [0, 11, 11], [7, 8, 9]], dtype=torch.int32)
    g = torch.randn((5, 3), generator=torch.Generator().manual_seed(5))
    got = run(l.cuda(), ids.cuda(), g.cuda(), score, renorm, 1.0)
    z = l.double().requires_grad_(True)
    s = torch.softmax(z, 1) if score == "softmax" else torch.sigmoid(z)
    w = s.gather(1, ids.long())
    if renorm:
        w = w / w.sum(1, keepdim=True)
    (want,) = torch.autograd.grad((w * g.double()).sum(), z)
    mag = 2 * g.abs().double().sum(1, keepdim=True)
    assert bool((torch.from_numpy(got) - want).abs().le(4 * W * mag).all())
