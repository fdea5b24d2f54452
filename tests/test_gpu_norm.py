"""The norms around a block and their gradients, against a plain implementation in 64 bits.

Bars: half a step of the result's type, and C * 2^-24 of the terms' absolute values for fp32 arithmetic, C = 64 covering
a row's sums (at most 32 in a thread, ten steps of the tree, the division and square root); a sum over rows adds one
2^-24 of its terms for each addition."""
import pytest
import torch

from combine_moe_layout_gb300 import _binding as B
from tests.gpu_common import require_gpu

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
C = 64 * 2.0 ** -24
GATES = [B.MOE_GATE_NONE, B.MOE_GATE_ROW, B.MOE_GATE_CHANNEL]


def half(t):
    return torch.finfo(t.dtype).eps / 2


class Case:
    def __init__(self, T, H, fp32, gate, post, block=True, seed=0, eps=1e-6, alpha=0.5):
        require_gpu()
        g = torch.Generator(device=DEV).manual_seed(seed)
        st = torch.float32 if fp32 else torch.bfloat16
        self.T, self.H, self.eps, self.alpha, self.kind = T, H, eps, alpha, gate

        def normal(*shape, dtype=torch.float32, scale=1.0, mean=0.0):
            return (torch.randn(shape, generator=g, device=DEV) * scale + mean).to(dtype)

        self.x = normal(T, H, dtype=st, scale=2.0)
        self.o = normal(T, H, dtype=torch.bfloat16) if block else None
        self.w_pre = normal(H, scale=0.3, mean=1.0)
        self.w_post = normal(H, scale=0.3, mean=1.0) if post else None
        self.gate = None if gate == B.MOE_GATE_NONE else normal(T if gate == B.MOE_GATE_ROW else H)
        self.r, self.n = torch.zeros_like(self.x), torch.zeros((T, H), dtype=torch.bfloat16, device=DEV)
        self.grad_r, self.grad_n = normal(T, H, dtype=st), normal(T, H, dtype=torch.bfloat16)
        self.desc = B.MoeNormDesc(T, H, int(fp32), gate, eps, alpha)
        self.err = torch.zeros(1, dtype=torch.int32, device=DEV)

    def g64(self):
        if self.gate is None:
            return 1.0
        return self.gate.double()[:, None] if self.kind == B.MOE_GATE_ROW else self.gate.double()

    def forward(self, r="own"):
        B.moe_norm(self.desc, self.x, self.o, self.w_post, self.gate, self.w_pre, self.r if r == "own" else r, self.n,
                   self.err)

    def formula(self, x, o, w_post, gate, w_pre):
        b = 0.0
        if o is not None:
            b = o
            if w_post is not None:
                b = b / (b.square().mean(1, keepdim=True) + self.eps).sqrt() * w_post
            if gate is not None:
                b = b * (gate[:, None] if self.kind == B.MOE_GATE_ROW else gate)
        r = x + self.alpha * b
        return r, r / (r.square().mean(1, keepdim=True) + self.eps).sqrt() * w_pre

    def wide(self):
        return [t.double() if t is not None else None for t in (self.x, self.o, self.w_post, self.gate, self.w_pre)]

    def check_forward(self):
        x, o, wp, g, w = self.wide()
        r, n = self.formula(x, o, wp, g, w)
        er = C * (x.abs() + (r - x).abs())
        assert bool(((self.r.double() - r).abs() <= half(self.r) * r.abs() + er).all())
        scale = (n / r).abs().nan_to_num(0.0)
        assert bool(((self.n.double() - n).abs() <= half(self.n) * n.abs() + 2 * C * n.abs() + 2 * er * scale).all())

    def backward(self, with_r=True):
        T, H = self.T, self.H
        self.gx = torch.full_like(self.x, 9.0)
        self.go = torch.full_like(self.o, 9.0) if self.o is not None else None
        self.gwp = torch.full((H,), 9.0, device=DEV) if self.w_post is not None else None
        self.gg = torch.full_like(self.gate, 9.0) if self.gate is not None else None
        self.gw = torch.full((H,), 9.0, device=DEV)
        work = torch.full((max(1, B.moe_norm_workspace(self.desc)),), 0xff, dtype=torch.uint8, device=DEV)
        B.moe_norm_grad(self.desc, self.x, self.o, self.w_post, self.gate, self.w_pre, self.grad_r if with_r else None,
                        self.grad_n, self.gx, self.go, self.gwp, self.gg, self.gw, work, self.err)

    def check_backward(self, with_r=True):
        """x is the stream that was kept. By autograd of the formula; the bars' terms with absolute values."""
        x, o, wp, g, w = self.wide()
        r = x
        dn, d0 = self.grad_n.double(), self.grad_r.double() * with_r
        leaves = [t.requires_grad_(True) for t in (o, wp, g, w) if t is not None]
        r0, _ = self.formula(torch.zeros_like(x), o, wp, g, w)
        x = (x - r0.detach()).requires_grad_(True)
        rr, nn = self.formula(x, o, wp, g, w)
        grads = list(torch.autograd.grad((rr * d0).sum() + (nn * dn).sum(), [x] + leaves, allow_unused=True))
        dx = grads.pop(0)
        with torch.no_grad():
            q = 1 / (r.square().mean(1, keepdim=True) + self.eps).sqrt()
            hat = r * q
            part = q * ((dn * w).abs() + hat.abs() * (dn * w * hat).abs().mean(1, keepdim=True))
            ex = C * (d0.abs() + 2 * part)  # of dr before it is rounded
            assert bool(((self.gx.double() - dx).abs() <= half(self.gx) * dx.abs() + ex).all())
            tall = dx.abs() + d0.abs() + part  # the sizes of what dr is made of
            if o is not None:
                do = grads.pop(0)
                p = 1 / (o.square().mean(1, keepdim=True) + self.eps).sqrt() if wp is not None else 1.0
                c = (wp if wp is not None else 1.0)
                gk = self.g64()
                t = abs(self.alpha) * (gk * c if torch.is_tensor(gk) or torch.is_tensor(c) else torch.ones_like(r)).abs() * tall
                ohat = o * p
                mean = (t * ohat.abs()).mean(1, keepdim=True) if wp is not None else 0.0
                eo = 4 * C * p * (t + ohat.abs() * mean)
                assert bool(((self.go.double() - do).abs() <= half(self.go) * do.abs() + eo).all())
                s = abs(self.alpha) * tall * ohat.abs()
                n = self.T + 64
                if wp is not None:
                    dwp = grads.pop(0)
                    sg = (s * (gk.abs() if torch.is_tensor(gk) else 1.0)).sum(0)
                    assert bool(((self.gwp.double() - dwp).abs() <= (4 * C + n * 2.0 ** -24) * sg).all())
                if g is not None:
                    dg = grads.pop(0)
                    sb = s * (wp.abs() if wp is not None else 1.0)
                    terms = sb.sum(1) if self.kind == B.MOE_GATE_ROW else sb.sum(0)
                    assert bool(((self.gg.double() - dg).abs() <= (8 * C + n * 2.0 ** -24) * terms).all())
            dw = grads.pop(0)
            assert bool(((self.gw.double() - dw).abs() <= (2 * C + (self.T + 64) * 2.0 ** -24)
                         * (dn * hat).abs().sum(0)).all())


SHAPES = [(1, 8), (1, 7168), (3, 128), (5, 1000), (333, 264), (700, 1024), (2, 4104), (3, 8192), (2, 16384), (1, 32768),
          (1300, 40)]


@pytest.mark.parametrize("T,H", SHAPES)
@pytest.mark.parametrize("fp32", [False, True])
@pytest.mark.parametrize("gate", GATES)
@pytest.mark.parametrize("post", [False, True])
def test_forward_and_gradients(T, H, fp32, gate, post):
    c = Case(T, H, fp32, gate, post)
    c.forward()
    c.check_forward()
    c.backward()
    c.check_backward()
    assert B.moe_get_error(c.err) == B.MOE_OK


@pytest.mark.parametrize("fp32", [False, True])
def test_no_block_before_it(fp32):
    c = Case(77, 520, fp32, B.MOE_GATE_NONE, False, block=False)
    c.forward(r=None)
    c.r.copy_(c.x)
    c.check_forward()
    c.backward()
    c.check_backward()
    c.backward(with_r=False)
    c.check_backward(with_r=False)


@pytest.mark.parametrize("fp32", [False, True])
def test_results_in_the_inputs_places(fp32):
    c = Case(50, 1000, fp32, B.MOE_GATE_ROW, True)
    c.forward()
    c.backward()
    r, gx, go = c.r.clone(), c.gx.clone(), c.go.clone()
    work = torch.empty(B.moe_norm_workspace(c.desc), dtype=torch.uint8, device=DEV)
    kept = c.x.clone()
    B.moe_norm(c.desc, c.x, c.o, c.w_post, c.gate, c.w_pre, c.x, c.n, c.err)
    assert torch.equal(c.x, r)
    for into in (c.grad_n.clone(), c.o.clone()):
        dr, dn = c.grad_r.clone(), c.grad_n
        o = c.o
        if bool(torch.equal(into, c.o)):
            o = into
        else:
            dn = into
        B.moe_norm_grad(c.desc, kept, o, c.w_post, c.gate, c.w_pre, dr, dn, dr, into, c.gwp, c.gg, c.gw, work, c.err)
        assert torch.equal(dr, gx) and torch.equal(into, go)


def test_zero_rows_of_a_block_and_of_the_stream():
    """A block that put out nothing adds nothing; the norm of a row of zeros is zero."""
    c = Case(9, 256, True, B.MOE_GATE_CHANNEL, True)
    c.o[3] = 0
    c.x[5] = 0
    c.o[5] = 0
    c.forward()
    c.check_forward()
    assert torch.equal(c.r[3], c.x[3]) and not c.n[5].any()


def test_what_is_not_finite_stays_in_its_row():
    c = Case(20, 264, False, B.MOE_GATE_ROW, True)
    c.x[4, 7] = float("nan")
    c.o[6, 0] = float("inf")
    c.forward()
    keep = [i for i in range(20) if i not in (4, 6)]
    assert bool(torch.isfinite(c.n[keep]).all()) and bool(torch.isfinite(c.r[keep]).all())
    assert bool(torch.isnan(c.n[4]).all())


def test_no_rows():
    c = Case(0, 128, False, B.MOE_GATE_CHANNEL, True)
    c.forward()
    c.backward()
    assert not c.gw.any() and not c.gwp.any() and not c.gg.any()
    assert B.moe_get_error(c.err) == B.MOE_OK


def test_gradient_against_differences():
    """sum(gradient * direction) against the slope of the 64-bit formula: fp32 stream, so that only grad_o is rounded
    (2^-8 of its terms, in the 2-norm with a factor of 4)."""
    c = Case(31, 200, True, B.MOE_GATE_CHANNEL, True)
    x0, o, wp, g, w = c.wide()
    r, _ = c.formula(x0, o, wp, g, w)
    kept = Case(31, 200, True, B.MOE_GATE_CHANNEL, True)
    kept.x = r.float()
    kept.backward()
    args = [r.float().double() - (r - x0), o, wp, g, w]

    def loss(a):
        rr, nn = c.formula(*a)
        return float((rr * c.grad_r.double()).sum() + (nn * c.grad_n.double()).sum())

    gen = torch.Generator(device=DEV).manual_seed(8)
    for i, grad in enumerate([kept.gx, kept.go, kept.gwp, kept.gg, kept.gw]):
        d = torch.randn(args[i].shape, generator=gen, device=DEV, dtype=torch.float64)
        step = 1e-5
        ends = [loss([t + s * step * d if j == i else t for j, t in enumerate(args)]) for s in (1, -1)]
        slope, terms = (ends[0] - ends[1]) / (2 * step), grad.double() * d
        bar = (4 * 2.0 ** -8 if i == 1 else 1e-4) * float(terms.norm()) + 1e-6 * abs(slope) + 1e-5
        assert abs(float(terms.sum()) - slope) <= bar, i


def test_captured_and_replayed():
    c = Case(300, 1000, False, B.MOE_GATE_CHANNEL, True)
    c.forward()
    c.backward()
    want = [t.clone() for t in (c.r, c.n, c.gx, c.go, c.gwp, c.gg, c.gw)]
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.forward()
        c.backward()
    for _ in range(2):
        for t in (c.r, c.n):
            t.fill_(3)
        g.replay()
        torch.cuda.synchronize()
        for got, w in zip((c.r, c.n, c.gx, c.go, c.gwp, c.gg, c.gw), want):
            assert torch.equal(got, w)
