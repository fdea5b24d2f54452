"""The layer of one device in training, as a model runs it: norm, router, experts beside a dense block, and the next
norm with a gate and the residual stream; forward and backward, against autograd in 64 bits.

Bars in the 2-norm of each result: every bf16 rounding on the way (n, h, the experts' rows, their sum, and as many on
the way back) leaves at most 2^-8 of the norm of what it rounds, and a feed-forward block, with two factors that are
linear in its input, at most doubles a relative error: 16 times 2^-8 for a result of the whole way there and back. The
reference takes the layer's own choice of experts, and its projections at the values that were kept."""
from __future__ import annotations

import pytest
import torch

from combine_moe_layout_gb300 import _binding as B
from combine_moe_layout_gb300 import pipeline as P
from combine_moe_layout_gb300 import workloads as wl
from gpu_common import require_gpu

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


class Step:
    def __init__(self, T=150, H=256, E=8, k=2, I=384, masked=True, seed=1):
        require_gpu()
        g = torch.Generator().manual_seed(seed)

        def normal(*shape, scale=1.0, dtype=torch.bfloat16, mean=0.0):
            return (torch.randn(shape, generator=g) * scale + mean).to(dtype).to(DEV)

        f32 = torch.float32
        self.T, self.H, self.E, self.k, self.I, self.alpha = T, H, E, k, I, 0.5
        self.layer = P.LocalMoe(T, H, E, k, B.MoeGateOpts(B.MOE_SCORE_SOFTMAX, 1, 0, 0, 0, 0, 1.0), DEV, I)
        self.x = normal(T, H, dtype=f32)
        self.w1, self.w2, self.wp = (normal(H, scale=0.2, dtype=f32, mean=1.0) for _ in range(3))
        self.gate = normal(H, scale=0.5, dtype=f32)
        self.router = normal(H, E, scale=H ** -0.5, dtype=f32)
        self.weights = wl.ExpertWeights(I, normal(E, I, H, scale=H ** -0.5), normal(E, I, H, scale=H ** -0.5),
                                        normal(E, H, I, scale=I ** -0.5))
        self.dw = (normal(I, H, scale=H ** -0.5), normal(I, H, scale=H ** -0.5), normal(H, I, scale=I ** -0.5))
        self.mask = torch.zeros((T, E), device=DEV)
        if masked:
            self.mask[7] = -float("inf")        # a token that no expert takes
            self.mask[:, 3] = -float("inf")     # an expert without tokens
        self.gr, self.gn = normal(T, H, dtype=f32), normal(T, H)

    def forward(self, save):
        m = self.layer
        _, self.n1 = m.norm(self.x, self.w1)
        self.logits = self.n1.float() @ self.router + self.mask
        self.out = m.forward(self.n1, self.logits, self.weights, save=save)
        self.shared, self.kept = m.dense(self.n1, *self.dw, save=save)
        self.o = self.out + self.shared
        return m.norm(self.x, self.w2, self.o, self.wp, self.gate, alpha=self.alpha)

    def backward(self, r):
        m = self.layer
        g = m.norm_grad(r, self.gn, self.w2, self.gr, self.o, self.wp, self.gate, alpha=self.alpha)
        gn_moe, gl = m.backward(g.o, self.logits, self.weights)
        gn_dense, *gdw = m.dense_grad(self.kept, self.n1, *self.dw, g.o)
        gl = gl.nan_to_num(0.0)
        gn1 = (gn_moe.float() + gn_dense.float() + gl @ self.router.t()).to(torch.bfloat16)
        first = m.norm_grad(self.x, gn1, self.w1, g.x)
        return {"x": first.x, "w1": first.w_pre, "w2": g.w_pre, "wp": g.w_post, "gate": g.gate,
                "router": self.n1.float().t() @ gl, "w_gate": m.grad_w_gate, "w_up": m.grad_w_up,
                "w_down": m.grad_w_down, "d_gate": gdw[0], "d_up": gdw[1], "d_down": gdw[2]}


def kept_values(k):
    if k.gate_scales is None:
        return k.gate.double(), k.up.double()
    return tuple(t.view(torch.float8_e4m3fn).double() * s.double().repeat_interleave(128, 1)
                 for t, s in ((k.gate, k.gate_scales), (k.up, k.up_scales)))


def block(x, wg, wu, wd, kept):
    """The block's value, with gradients as at the kept projections."""
    g, u = x @ wg.t(), x @ wu.t()
    gk, uk = g + (kept[0] - g).detach(), u + (kept[1] - u).detach()

    def f(g, u):
        return (g * torch.sigmoid(g) * u) @ wd.t()

    at = f(gk, uk)
    return at + (f(g, u) - at).detach()


def norm64(x, w):
    return x / (x.square().mean(1, keepdim=True) + 1e-6).sqrt() * w


def reference(s: Step):
    names = ("x", "w1", "w2", "wp", "gate", "router")
    t = {n: getattr(s, n).double().requires_grad_(True) for n in names}
    e = {n: getattr(s.weights, n).double().requires_grad_(True) for n in ("w_gate", "w_up", "w_down")}
    d = {n: w.double().requires_grad_(True) for n, w in zip(("d_gate", "d_up", "d_down"), s.dw)}
    m = s.layer
    n1 = norm64(t["x"], t["w1"])
    logits = n1 @ t["router"] + s.mask.double()
    idx, tok = m.topk_idx.long(), m.tok_packed.long()
    probs = torch.softmax(logits.masked_fill(idx[:, :1] < 0, 0.0), 1)
    w = probs.gather(1, idx.clamp(min=0)) * (idx >= 0)
    w = w / w.sum(1, keepdim=True).clamp(min=1e-30)
    gk, uk = kept_values(m.kept)
    out = torch.zeros_like(n1)
    for ex in range(s.E):
        at = (idx == ex).nonzero()
        if len(at) == 0:
            continue
        rows = tok[at[:, 0], at[:, 1]]
        y = block(n1[at[:, 0]], e["w_gate"][ex], e["w_up"][ex], e["w_down"][ex], (gk[rows], uk[rows]))
        out = out.index_add(0, at[:, 0], w[at[:, 0], at[:, 1]][:, None] * y)
    o = out + block(n1, d["d_gate"], d["d_up"], d["d_down"], kept_values(s.kept))
    r = t["x"] + s.alpha * t["gate"] * norm64(o, t["wp"])
    n2 = norm64(r, t["w2"])
    leaves = {**t, **e, **d}
    grads = torch.autograd.grad((r * s.gr.double()).sum() + (n2 * s.gn.double()).sum(), list(leaves.values()))
    return r.detach(), n2.detach(), dict(zip(leaves, grads))


def near(name, got, want, times):
    off = float((got.double() - want).norm() / want.norm())
    assert off <= times * 2.0 ** -8, (name, off)


@pytest.mark.parametrize("save", ["bf16", "fp8"])
def test_a_step_forward_and_backward(save):
    s = Step()
    r, n2 = s.forward(save)
    got = s.backward(r)
    assert s.layer.error() == B.MOE_OK
    wr, wn, want = reference(s)
    near("r", r, wr, 8)
    near("n2", n2, wn, 8)
    for name, w in want.items():
        near(name, got[name], w, 16)
    assert not s.layer.grad_w_gate[3].any() and not s.layer.grad_w_down[3].any()


def test_a_forward_that_keeps_has_the_results_of_one_that_does_not():
    """To a rounding: both sum the same products in fp32, by the same kernel's tiles in another order."""
    s = Step(masked=False)
    s.forward("bf16")
    y = s.out.clone()
    plain = s.layer.forward(s.n1, s.logits, s.weights)
    near("out", y, plain.double(), 1)


def test_captured_on_another_stream_and_replayed():
    s = Step(T=70)
    r, n2 = s.forward("fp8")
    want = {k: v.clone() for k, v in s.backward(r).items()}
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        s.backward(s.forward("fp8")[0])  # the first call on this stream
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        r, n2 = s.forward("fp8")
        got = s.backward(r)
    for _ in range(2):
        g.replay()
        torch.cuda.synchronize()
        for name, w in want.items():
            assert torch.equal(got[name], w), name
    assert s.layer.error() == B.MOE_OK


@pytest.mark.parametrize("T", [1, 16, 40])
def test_a_dense_block_for_few_tokens(T):
    s = Step(T=T, masked=False)
    y, kept = s.layer.dense(s.gn, *s.dw)
    assert kept is None and s.layer.error() == B.MOE_OK
    g = s.gn.double() @ s.dw[0].double().t()
    near("y", y, (g * torch.sigmoid(g) * (s.gn.double() @ s.dw[1].double().t())) @ s.dw[2].double().t(), 4)


def test_backward_does_not_go_by_what_an_earlier_forward_kept():
    s = Step(T=20, masked=False)
    r, _ = s.forward("bf16")
    s.layer.forward(s.n1, s.logits, s.weights)
    with pytest.raises(ValueError, match="follows a forward with save"):
        s.backward(r)
