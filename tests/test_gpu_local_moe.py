"""The layer of one device (pipeline.LocalMoe): router, sort, experts, way back
and shared projection together.

The routed output has to be the dispatch path's, bit for bit: the same rows meet
the same kernels in the same order. The gradients are held against autograd in 64
bits of the formula out_t = sum_j w_tj x_t f_e (experts that scale by a power of
two, so that they round nothing): bf16 roundings of grad_y and of grad_x leave
2^-7 of the sum of magnitudes; the weights' gradient sums H products of bf16
values in fp32, (H / 32 + 24) 2^-24 of their magnitudes, and the logits' adds
the gate's own bar, below 2^-14 of the largest."""
from __future__ import annotations

import pytest
import torch

from combine_moe_layout_gb300 import _binding as B
from combine_moe_layout_gb300 import pipeline as P
from combine_moe_layout_gb300 import workloads as wl
from gpu_common import require_gpu

pytestmark = pytest.mark.gpu


def opts(score=B.MOE_SCORE_SOFTMAX):
    return B.MoeGateOpts(score, 1, 0, 0, 0, 0, 1.0)


def test_forward_is_the_dispatch_path():
    require_gpu()
    T, H, E, k, I = 150, 256, 8, 2, 384
    w = wl.custom("local", num_ranks=1, tokens_per_rank=T, hidden=H, num_experts=E, topk=k, max_m=T, intermediate=I,
                  x_dist="normal")
    g = torch.Generator().manual_seed(1)
    x = torch.randn((T, H), generator=g).to(torch.bfloat16).cuda()
    logits = torch.randn((T, E), generator=g)
    logits[7] = -float("inf")        # a token that no expert takes
    logits[9, 1:] = -float("inf")    # and one with a single expert
    logits = logits.cuda()
    wts = wl.expert_weights(w, "cuda:0")
    layer = P.LocalMoe(T, H, E, k, opts(), "cuda:0", I)
    out = layer.forward(x, logits, wts)
    assert layer.error() == B.MOE_OK

    step = P.MoeStep(w, "cuda:0")
    d = P.DeviceInputs(layer.topk_idx.view(1, T, k), layer.topk_weights.view(1, T, k), x.view(1, T, H), None)
    step.reset()
    step.layout_dispatch(d)
    packed = B.allocate_packed(step.desc, "cuda:0")
    step.recv(packed)
    h = torch.empty((T * k, I), dtype=torch.bfloat16, device="cuda:0")
    y = torch.empty((T * k, H), dtype=torch.bfloat16, device="cuda:0")
    step.expert_mlp(wts, packed, h, y)
    step.combine_packed(d, y, packed)
    assert step.error() == B.MOE_OK
    assert torch.equal(layer.region_offsets, packed.region_offsets)
    assert torch.equal(out, step.buf.out.view(T, H))
    assert bool((out[7] == 0).all()) and float(layer.topk_weights[9, 0]) == 1.0


@pytest.mark.parametrize("score", [B.MOE_SCORE_SOFTMAX, B.MOE_SCORE_SIGMOID])
def test_backward_against_autograd(score):
    require_gpu()
    T, H, E, k = 70, 264, 12, 3
    g = torch.Generator().manual_seed(2)
    x = torch.randn((T, H), generator=g).to(torch.bfloat16).cuda()
    logits = torch.randn((T, E), generator=g).cuda()
    go = torch.randn((T, H), generator=g).to(torch.bfloat16).cuda()
    fac = torch.tensor([2.0 ** (e % 4 - 1) for e in range(E)], device="cuda:0")
    layer = P.LocalMoe(T, H, E, k, opts(score), "cuda:0")
    layer.route(logits)
    layer.sort(x)
    expert = torch.searchsorted(layer.region_offsets[1:].long(), torch.arange(T * k, device="cuda:0"), right=True)
    scale = fac[expert][:, None].to(torch.bfloat16)
    torch.mul(layer.packed_x, scale, out=layer.packed_y)
    layer.unsort()
    gx, gl = layer.backward(go, logits, lambda px, off, gy: gy * scale)
    assert layer.error() == B.MOE_OK

    xd, ld = x.double().requires_grad_(True), logits.double().requires_grad_(True)
    s = torch.softmax(ld, 1) if score == B.MOE_SCORE_SOFTMAX else torch.sigmoid(ld)
    idx = layer.topk_idx.long()
    wt = s.gather(1, idx)
    wt = wt / wt.sum(1, keepdim=True)
    coef = (wt * fac.double()[idx]).sum(1, keepdim=True)
    wx, wl_ = torch.autograd.grad((coef * xd * go.double()).sum(), (xd, ld))
    mag = (wt * fac.double()[idx]).sum(1, keepdim=True).detach() * go.double().abs()
    assert bool(((gx.double() - wx).abs() <= 2.0 ** -7 * mag).all())
    dots = (x.double().abs() * go.double().abs()).sum(1, keepdim=True) * fac.double().max()
    bar = ((H / 32 + 24) * 2.0 ** -24 + 2.0 ** -14) * dots
    assert bool(((gl.double() - wl_).abs() <= bar).all())


def test_shared_projection_beside_the_experts():
    require_gpu()
    T, H, N, r, A = 90, 256, 512, 16, 5
    g = torch.Generator().manual_seed(3)

    def draw(*shape, scale=1.0):
        return (torch.randn(shape, generator=g) * scale).to(torch.bfloat16).cuda()

    x, w, la, lb = draw(T, H), draw(N, H, scale=H ** -0.5), draw(A, r, H, scale=H ** -0.5), draw(A, N, r, scale=r ** -0.5)
    ids = torch.randint(-1, A, (T,), generator=g, dtype=torch.int32).cuda()
    layer = P.LocalMoe(T, H, 4, 1, opts(), "cuda:0")
    y = layer.shared(x, w, la, lb, None, ids)
    assert layer.error() == B.MOE_OK
    want = x.double() @ w.double().t()
    for a in range(A):
        t = (ids == a).nonzero().view(-1)
        want[t] += (x[t].double() @ la[a].double().t()) @ lb[a].double().t()
    # one bf16 rounding of y and one of u, with fp32 sums far below: 2^-7 of the magnitudes that are added
    mag = x.double().abs() @ w.double().abs().t() * 2.0 ** -8
    assert bool(((y.double() - want).abs() <= 2.0 ** -7 * want.abs() + mag).all())


def test_shared_takes_another_shape():
    """A second projection of another width and rank: its own buffers, and the first one's result stays."""
    require_gpu()
    g = torch.Generator().manual_seed(4)
    layer = P.LocalMoe(20, 128, 4, 1, opts(), "cuda:0")
    x = torch.randn((20, 128), generator=g).to(torch.bfloat16).cuda()
    ids = (torch.arange(20) % 3).to(torch.int32).cuda()
    first = None
    for N, r in ((64, 8), (264, 40), (264, 16)):
        w = torch.randn((N, 128), generator=g).to(torch.bfloat16).cuda()
        la = torch.randn((3, r, 128), generator=g).to(torch.bfloat16).cuda()
        lb = torch.zeros((3, N, r), dtype=torch.bfloat16, device="cuda")
        y = layer.shared(x, w, la, lb, None, ids)
        assert layer.error() == B.MOE_OK and y.shape == (20, N) and layer.u.shape == (20, r)
        want = x.double() @ w.double().t()
        bar = 2.0 ** -8 * want.abs() + 128 * 2.0 ** -23 * (x.double().abs() @ w.double().abs().t())
        assert bool(((y.double() - want).abs() <= bar).all())
        if first is None:
            first, kept = y, y.clone()
    assert torch.equal(first, kept)
