"""The gated feed-forward block, what it keeps, and its gradients, against a plain implementation in 64 bits.

Bars, element by element: half a step of each rounding to bf16 (2^-8 of the value), carried through the product that
follows with absolute values, and (terms + 16) * 2^-23 of the sum of the terms' absolute values for a sum in fp32
(each of its steps is off by at most one unit in the last place, 2^-23, of what has been summed)."""
import math

import pytest
import torch

from combine_moe_layout_gb300 import _binding as B
from tests.gpu_common import require_gpu

pytestmark = pytest.mark.gpu

U = 2.0 ** -8  # half a step of bf16
SLACK = 1.02   # second-order terms: a rounding of a rounded value
DEV = "cuda:0"


def gam(n):
    return (n + 16) * 2.0 ** -23


def act64(g, act):
    if act == B.MOE_ACT_SILU:
        s = torch.sigmoid(g)
        return g * s, s * (1 + g * (1 - s))
    k = math.sqrt(2 / math.pi)
    t = torch.tanh(k * (g + 0.044715 * g ** 3))
    return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * k * (1 + 3 * 0.044715 * g * g)


class Case:
    """Inputs and buffers of a block; `counts` rows of each expert, `behind` rows behind the last one."""

    def __init__(self, counts, H, I, act=B.MOE_ACT_SILU, save=B.MOE_SAVE_NONE, behind=0, ranks=1, num_sms=0, seed=0,
                 dense=False):
        require_gpu()
        self.counts, self.H, self.I, self.E, self.act, self.save = counts, H, I, len(counts), act, save
        self.n = sum(counts)
        self.rows = self.n + behind
        g = torch.Generator(device=DEV).manual_seed(seed)

        def normal(*shape, scale=1.0):
            return (torch.randn(shape, generator=g, device=DEV) * scale).to(torch.bfloat16)

        self.normal = normal
        starts = [0]
        for c in counts:  # an expert's rows in `ranks` regions
            for r in range(ranks):
                starts.append(starts[-1] + (c // ranks if r + 1 < ranks else c - (ranks - 1) * (c // ranks)))
        self.offsets = None if dense else torch.tensor(starts, dtype=torch.int32, device=DEV)
        self.x = normal(self.rows, H)
        self.w_gate, self.w_up = normal(self.E, I, H, scale=H ** -0.5), normal(self.E, I, H, scale=H ** -0.5)
        self.w_down = normal(self.E, H, I, scale=I ** -0.5)
        self.err = torch.zeros(1, dtype=torch.int32, device=DEV)
        self.desc = B.MoeFfnDesc(self.rows, H, I, self.E, ranks, act, save, num_sms)
        self.h = torch.zeros((self.rows, I), dtype=torch.bfloat16, device=DEV)
        self.y = torch.full((self.rows, H), 7.0, dtype=torch.bfloat16, device=DEV)
        self.gate = self.up = self.gate_scales = self.up_scales = None
        if save != B.MOE_SAVE_NONE:
            t = torch.bfloat16 if save == B.MOE_SAVE_BF16 else torch.uint8
            self.gate, self.up = (torch.full((self.rows, I), 5, dtype=t, device=DEV) for _ in range(2))
        if save == B.MOE_SAVE_FP8:
            self.gate_scales, self.up_scales = (torch.full((self.rows, I // 128), 3.0, device=DEV) for _ in range(2))

    def runs(self):
        at = 0
        for e, c in enumerate(self.counts):
            yield e, at, at + c
            at += c

    def forward(self, stream=None):
        B.moe_ffn(self.desc, self.offsets, self.x, self.w_gate, self.w_up, self.w_down, self.h, self.y, self.gate,
                  self.gate_scales, self.up, self.up_scales, self.err, stream)

    def check_forward(self):
        assert B.moe_get_error(self.err) == B.MOE_OK
        for e, a, b in self.runs():
            x, wg, wu, wd = (t.double() for t in (self.x[a:b], self.w_gate[e], self.w_up[e], self.w_down[e]))
            g, u = x @ wg.t(), x @ wu.t()
            eg, eu = gam(self.H) * (x.abs() @ wg.abs().t()), gam(self.H) * (x.abs() @ wu.abs().t())
            if self.save == B.MOE_SAVE_BF16:
                assert bool(((self.gate[a:b].double() - g).abs() <= U * g.abs() + SLACK * eg).all())
                assert bool(((self.up[a:b].double() - u).abs() <= U * u.abs() + SLACK * eu).all())
            if self.save == B.MOE_SAVE_FP8:
                check_codes(self.gate[a:b], self.gate_scales[a:b], g, eg)
                check_codes(self.up[a:b], self.up_scales[a:b], u, eu)
            p, dp = act64(g, self.act)
            h = p * u
            eh = U * h.abs() + 1.13 * eg * u.abs() + p.abs() * eu + 2.0 ** -20 * (1 + g.abs()) * u.abs()
            y = h @ wd.t()
            bar = U * y.abs() + SLACK * (eh @ wd.abs().t() + gam(self.I) * (h.abs() @ wd.abs().t()))
            assert bool(((self.y[a:b].double() - y).abs() <= bar).all()), (e, (self.y[a:b].double() - y).abs().max())
        assert bool((self.y[self.n:] == 7.0).all())
        if self.save != B.MOE_SAVE_NONE:
            assert bool((self.gate[self.n:] == 5).all()) and bool((self.up[self.n:] == 5).all())
        if self.save == B.MOE_SAVE_FP8:
            assert bool((self.gate_scales[self.n:] == 3).all()) and bool((self.up_scales[self.n:] == 3).all())

    def keep_made(self):
        """What a forward would have kept, made here: any values, rows behind the last among them."""
        g, u = self.normal(self.rows, self.I, scale=1.5), self.normal(self.rows, self.I)
        if self.save == B.MOE_SAVE_FP8:
            for name, t in (("gate", g), ("up", u)):
                b = t.float().view(self.rows, -1, 128)
                s = b.abs().amax(2) / 448.0
                getattr(self, name).copy_((b / s[:, :, None]).to(torch.float8_e4m3fn).view(self.rows, -1)
                                          .view(torch.uint8))
                getattr(self, name + "_scales").copy_(s)
        else:
            self.gate, self.up = g, u
        self.grad_y = self.normal(self.rows, self.H)

    def kept(self, name, a, b):
        t = getattr(self, name)[a:b]
        if self.save == B.MOE_SAVE_BF16:
            return t.double()
        s = getattr(self, name + "_scales")[a:b].double()
        return t.view(torch.float8_e4m3fn).double() * s.repeat_interleave(128, 1)

    def backward(self, weights=True, stream=None, reuse=False):
        if not reuse:
            self.hg, self.gg, self.gu = (torch.zeros((self.rows, self.I), dtype=torch.bfloat16, device=DEV)
                                         for _ in range(3))
            self.gx = torch.full((self.rows, self.H), 7.0, dtype=torch.bfloat16, device=DEV)
            self.gw = [torch.full_like(t, 9.0) for t in (self.w_gate, self.w_up, self.w_down)] if weights else [None] * 3
        B.moe_ffn_grad(self.desc, self.offsets, self.x, self.gate, self.gate_scales, self.up, self.up_scales, self.w_gate,
                       self.w_up, self.w_down, self.grad_y, self.hg, self.gg, self.gu, self.gx, *self.gw, self.err,
                       stream)

    def check_backward(self, experts=None):
        assert B.moe_get_error(self.err) == B.MOE_OK
        for e, a, b in self.runs():
            if experts is not None and e not in experts:
                continue
            x, dy, wg, wu, wd = (t.double() for t in (self.x[a:b], self.grad_y[a:b], self.w_gate[e], self.w_up[e],
                                                      self.w_down[e]))
            g, u = self.kept("gate", a, b), self.kept("up", a, b)
            p, dp = act64(g, self.act)
            dh, eh = dy @ wd, gam(self.H) * (dy.abs() @ wd.abs())
            tiny = 2.0 ** -20 * (1 + g.abs())  # fp32 values of act and its derivative
            dg, du, h = dh * u * dp, dh * p, p * u
            edg = U * dg.abs() + (u * dp).abs() * eh + tiny * (dh * u).abs()
            edu = U * du.abs() + p.abs() * eh + tiny * dh.abs()
            ehid = U * h.abs() + tiny * u.abs()

            def near(got, want, err, terms, n):
                bar = U * want.abs() + SLACK * (err + gam(n) * terms)
                d = (got.double() - want).abs()
                assert bool((d <= bar).all()), (e, a, b, float((d - bar).max()))

            near(self.gx[a:b], dg @ wg + du @ wu, edg @ wg.abs() + edu @ wu.abs(), dg.abs() @ wg.abs() + du.abs() @ wu.abs(),
                 2 * self.I)
            if self.gw[0] is None:
                continue
            near(self.gw[0][e], dg.t() @ x, edg.t() @ x.abs(), dg.abs().t() @ x.abs(), b - a)
            near(self.gw[1][e], du.t() @ x, edu.t() @ x.abs(), du.abs().t() @ x.abs(), b - a)
            near(self.gw[2][e], dy.t() @ h, dy.abs().t() @ ehid, dy.abs().t() @ h.abs(), b - a)
        assert bool((self.gx[self.n:] == 7.0).all())


def check_codes(codes, scales, want, err):
    """e4m3 codes and scales of `want`, itself known to `err`: half a step of e4m3 (2^-4 of a normal value, 2^-10 of
    the scale below it), the scale amax / 448 as near as the values are."""
    n = want.shape[0]
    if n == 0:
        return
    w, er = want.view(n, -1, 128), err.view(n, -1, 128)
    s = scales.double()
    amax = w.abs().amax(2)
    assert bool(((s - amax / 448).abs() <= er.amax(2) / 448 + 2.0 ** -22 * amax / 448).all())
    got = codes.view(torch.float8_e4m3fn).double().view(n, -1, 128) * s[:, :, None]
    bar = 2.0 ** -4 * w.abs() + 2.0 ** -10 * s[:, :, None] + SLACK * 2 * er + 2.0 ** -20 * w.abs()
    assert bool(((got - w).abs() <= bar).all())


SHAPES = [  # counts, H, I
    ([1], 256, 128), ([1], 8, 8), ([5], 72, 136), ([64], 128, 128), ([65], 264, 72), ([129], 64, 264),
    ([16], 264, 200), ([17], 264, 200), ([0, 9, 0, 3, 1], 1000, 712), ([200], 1000, 712), ([0, 3, 0, 130, 1, 64, 0], 328, 200), ([63, 64, 65, 127, 128, 129], 256, 384),
    ([700, 5], 512, 640), ([0, 0], 128, 128),
]


@pytest.mark.parametrize("counts,H,I", SHAPES)
@pytest.mark.parametrize("act", [B.MOE_ACT_SILU, B.MOE_ACT_GELU_TANH])
@pytest.mark.parametrize("save", [B.MOE_SAVE_NONE, B.MOE_SAVE_BF16])
def test_forward(counts, H, I, act, save):
    c = Case(counts, H, I, act, save, behind=3)
    c.forward()
    c.check_forward()


@pytest.mark.parametrize("counts,H,I", [([1], 128, 128), ([77], 328, 384), ([0, 3, 0, 130, 1, 64, 0], 256, 640)])
@pytest.mark.parametrize("act", [B.MOE_ACT_SILU, B.MOE_ACT_GELU_TANH])
def test_forward_keeps_8_bits(counts, H, I, act):
    c = Case(counts, H, I, act, B.MOE_SAVE_FP8, behind=2)
    c.forward()
    c.check_forward()


def test_forward_of_zero_rows_keeps_scale_one():
    c = Case([40], 128, 256, save=B.MOE_SAVE_FP8)
    c.x.zero_()
    c.forward()
    c.check_codes = None
    assert B.moe_get_error(c.err) == B.MOE_OK
    assert bool((c.gate_scales == 1).all()) and bool((c.up_scales == 1).all())
    assert not c.gate.any() and not c.up.any() and not c.y.any()


@pytest.mark.parametrize("counts,H,I", SHAPES)
@pytest.mark.parametrize("act", [B.MOE_ACT_SILU, B.MOE_ACT_GELU_TANH])
def test_gradients(counts, H, I, act):
    c = Case(counts, H, I, act, B.MOE_SAVE_BF16, behind=3, seed=1)
    c.keep_made()
    c.backward()
    c.check_backward()
    for e, n in enumerate(counts):
        if n == 0:
            assert not any(t[e].any() for t in c.gw)


@pytest.mark.parametrize("counts,H,I", [([1], 128, 128), ([77], 328, 384), ([0, 3, 0, 130, 1, 64, 0], 256, 640)])
@pytest.mark.parametrize("act", [B.MOE_ACT_SILU, B.MOE_ACT_GELU_TANH])
def test_gradients_from_8_bits(counts, H, I, act):
    c = Case(counts, H, I, act, B.MOE_SAVE_FP8, behind=2, seed=2)
    c.keep_made()
    c.backward()
    c.check_backward()


@pytest.mark.parametrize("ranks,num_sms", [(1, 1), (2, 7), (4, 0), (1, 10000)])
def test_regions_of_several_ranks_and_few_sms(ranks, num_sms):
    c = Case([70, 0, 201, 33], 264, 392, save=B.MOE_SAVE_BF16, behind=1, ranks=ranks, num_sms=num_sms)
    c.forward()
    c.check_forward()
    c.keep_made()
    c.backward()
    c.check_backward()


@pytest.mark.parametrize("n", [1, 40, 300])
def test_dense_without_offsets(n):
    c = Case([n], 392, 520, save=B.MOE_SAVE_BF16, dense=True)
    c.forward()
    c.check_forward()
    c.keep_made()
    c.backward(weights=False)
    c.check_backward()


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_what_is_not_finite_stays_in_its_expert(bad):
    """Rows of other experts and behind the last one share K blocks and tiles with an expert's own."""
    c = Case([37, 90, 70], 264, 136, save=B.MOE_SAVE_BF16, behind=9, seed=3)
    for t in (c.x, c.w_gate[1], c.w_up[1], c.w_down[1]):
        t[37:127 if t is c.x else None] = bad
    c.x[c.n:] = bad
    c.forward()
    torch.cuda.synchronize()
    assert bool(torch.isfinite(c.y[:37]).all()) and bool(torch.isfinite(c.y[127:]).all())
    c.keep_made()
    for t in (c.grad_y, c.gate, c.up):
        t[37:127] = bad
        t[c.n:] = bad
    c.backward()
    c.check_backward(experts=[0, 2])


def test_offsets_that_are_no_ranges_are_an_error_and_no_rows():
    c = Case([30, 30, 30], 128, 128, save=B.MOE_SAVE_BF16)
    c.offsets.copy_(torch.tensor([0, 30, 20, 1 << 20], dtype=torch.int32))
    c.forward()
    assert B.moe_get_error(c.err) == B.MOE_EINVAL
    assert bool((c.y[30:] == 7.0).all())
    c.keep_made()
    c.backward()
    assert B.moe_get_error(c.err) == B.MOE_EINVAL
    assert bool((c.gx[30:] == 7.0).all()) and not any(t[1:].any() for t in c.gw)


def test_offsets_that_are_no_ranges_of_few_rows():
    c = Case([5, 4, 3], 128, 128)
    c.offsets.copy_(torch.tensor([0, 5, 3, 1 << 20], dtype=torch.int32))
    c.forward()
    assert B.moe_get_error(c.err) == B.MOE_EINVAL
    assert bool((c.y[5:] == 7.0).all()) and bool((c.y[:5] != 7.0).any())


def test_no_rows():
    c = Case([0], 128, 128, save=B.MOE_SAVE_BF16)
    c.forward()
    c.keep_made()
    c.backward()
    assert B.moe_get_error(c.err) == B.MOE_OK
    assert not any(t.any() for t in c.gw)


def test_gradient_against_differences():
    """sum(gradient * direction) against the slope of the 64-bit forward, from bf16 values that the forward kept: the
    bar is the gradients' own roundings and those of what was kept, each 2^-8 of its terms."""
    c = Case([50, 21], 136, 200, act=B.MOE_ACT_GELU_TANH, save=B.MOE_SAVE_BF16, seed=4)
    c.forward()
    c.grad_y = c.normal(c.rows, c.H)
    c.backward()
    assert B.moe_get_error(c.err) == B.MOE_OK

    def loss(x, wg, wu, wd):
        total = 0.0
        for e, a, b in c.runs():
            h = act64(x[a:b] @ wg[e].t(), c.act)[0] * (x[a:b] @ wu[e].t())
            total = total + ((h @ wd[e].t()) * c.grad_y[a:b].double()).sum()
        return float(total)

    args = [t.double() for t in (c.x, c.w_gate, c.w_up, c.w_down)]
    g = torch.Generator(device=DEV).manual_seed(5)
    for i, grad in enumerate([c.gx] + c.gw):
        d = torch.randn(args[i].shape, generator=g, device=DEV, dtype=torch.float64) * args[i].std()
        step = 1e-5
        ends = [loss(*[t + s * step * d if j == i else t for j, t in enumerate(args)]) for s in (1, -1)]
        slope = (ends[0] - ends[1]) / (2 * step)
        got = float((grad.double() * d).sum())
        # roundings of kept values, intermediates and result are independent: four of 2^-8, in the 2-norm
        assert abs(got - slope) <= 4 * U * float((grad.double() * d).norm()) * 4 + 1e-6 * abs(slope), (i, got, slope)


def test_captured_and_replayed_beside_another_stream():
    c = Case([70, 9, 130], 264, 200, save=B.MOE_SAVE_BF16, behind=2)
    c.keep_made()
    c.forward()
    c.backward()
    torch.cuda.synchronize()
    want = [t.clone() for t in [c.y, c.gate, c.up, c.gx] + c.gw]
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        c.forward()
        c.backward(reuse=True)
    for t in [c.y, c.gate, c.up, c.gx] + c.gw:
        t.fill_(7)
    other = Case([70, 9, 130], 264, 200, save=B.MOE_SAVE_BF16, behind=2)
    torch.cuda.synchronize()
    g.replay()
    with torch.cuda.stream(s):
        other.forward()
    torch.cuda.synchronize()
    other.check_forward()
    for got, w in zip([c.y, c.gate, c.up, c.gx] + c.gw, want):
        assert torch.equal(got[:c.n] if got.shape[0] == c.rows else got, w[:c.n] if got.shape[0] == c.rows else w)
    assert B.moe_get_error(c.err) == B.MOE_OK


def off_by_16_bytes(t):
    """The same values in memory that begins on 16 bytes and not on 32."""
    e = 16 // t.element_size()
    room = torch.zeros(t.numel() + e, dtype=t.dtype, device=t.device)
    v = room[e:].view(t.shape)
    v.copy_(t)
    return v


@pytest.mark.parametrize("n", [5, 40, 300, 3000])
def test_matrices_that_begin_on_16_bytes(n):
    c = Case([n, 20], 256, 384, save=B.MOE_SAVE_BF16)
    for name in ("x", "w_gate", "w_up", "w_down", "h", "y", "gate", "up"):
        setattr(c, name, off_by_16_bytes(getattr(c, name)))
    c.forward()
    c.check_forward()
    c.keep_made()
    c.backward()
    for name in ("gate", "up", "grad_y", "hg", "gg", "gu", "gx"):
        setattr(c, name, off_by_16_bytes(getattr(c, name)))
    c.gw = [off_by_16_bytes(t) for t in c.gw]
    c.backward(reuse=True)
    c.check_backward()


@pytest.mark.parametrize("save", [B.MOE_SAVE_BF16, B.MOE_SAVE_FP8])
@pytest.mark.parametrize("counts,H,I", [([3000, 900], 512, 640), ([40] * 70, 256, 256)])
def test_many_tiles(counts, H, I, save):
    """More tiles than there are SMs: every CTA takes several."""
    c = Case(counts, H, I, save=save, behind=5, seed=6)
    c.forward()
    c.check_forward()
    c.keep_made()
    c.backward()
    c.check_backward()


def test_two_calls_at_once_on_two_streams():
    a = Case([70, 9, 130], 264, 200, save=B.MOE_SAVE_BF16, behind=2)
    b = Case([500, 300], 512, 392, save=B.MOE_SAVE_BF16, seed=7)
    for c in (a, b):
        c.keep_made()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        for c, s in zip((a, b), streams):
            with torch.cuda.stream(s):
                c.backward()
    torch.cuda.synchronize()
    a.check_backward()
    b.check_backward()


def test_results_do_not_depend_on_timing():
    c = Case([200, 37], 520, 392, save=B.MOE_SAVE_BF16)
    c.keep_made()
    first = None
    for _ in range(3):
        c.forward()
        c.gate, c.up = c.gate.clone(), c.up.clone()
        c.backward()
        got = [c.y[:c.n].clone(), c.gx[:c.n].clone()] + [t.clone() for t in c.gw]
        first = first or got
        assert all(torch.equal(x, y) for x, y in zip(got, first))


def test_the_first_call_of_a_size_in_a_capture():
    """Limits and numbers that are asked of the device once may be asked while a stream is captured."""
    c = Case([90], 1032, 264, save=B.MOE_SAVE_BF16, num_sms=90)
    c.keep_made()
    want = Case([90], 1032, 264, save=B.MOE_SAVE_BF16, num_sms=90)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        want.forward()
    g.replay()
    torch.cuda.synchronize()
    want.check_forward()
