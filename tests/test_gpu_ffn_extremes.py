"""The activations and their derivatives at every size that a bf16 projection has, from subnormals to the type's largest.

Widths of 8 with unit weights, so that every product has one term and each result shows one value. Bars: two roundings
to bf16 (h or dg, and the result: 2^-8 of the value each, 1.01 for their product), and 2^-20 (1 + |g|) for the fp32
arithmetic of act and act' (the block's own bar elsewhere), where |g| counts up to 100: beyond, both are g and 1, or 0,
to fp32."""
import pytest
import torch

from combine_moe_layout_gb300 import _binding as B
from test_gpu_ffn import DEV, U, Case, act64

pytestmark = pytest.mark.gpu
W = 8
TOP = float(torch.finfo(torch.bfloat16).max)
SIZES = [0.0, 1e-40, 1e-20, 0.5, 3.0, 9.0, 20.0, 60.0, 88.0, 104.0, 3e3, 1e7, 1e12, 1e13, 1.5e19, 3e19, 1e20, 1e30, TOP]
VALUES = [s * v for v in SIZES for s in (1.0, -1.0)]
ACTS = [B.MOE_ACT_SILU, B.MOE_ACT_GELU_TANH]


def unit():
    return torch.eye(W, dtype=torch.bfloat16, device=DEV)[None]


def near(got, want, g):
    bar = 2 * 1.01 * U * want.abs() + 2.0 ** -20 * (1 + g.abs().clamp(max=100.0))
    off = (got.double() - want).abs()
    assert bool((off <= bar).all()), [(float(g[i, j]), float(got[i, j]), float(want[i, j]))
                                      for i, j in (~(off <= bar)).nonzero()[:5].tolist()]


def of(c):
    """Each row of the case holds one of the values, the largest last, in each column."""
    v = torch.tensor(VALUES[-c.rows:], dtype=torch.float64, device=DEV).to(torch.bfloat16)
    return v[:, None].expand(-1, W).contiguous()


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("rows", [16, len(VALUES)])
def test_forward(act, rows):
    """rows: the form for few rows and tiles. x holds the row's value and a one: g and u."""
    c = Case([rows], W, W, act)
    v = of(c)
    c.x.zero_()
    c.x[:, 0], c.x[:, 1] = v[:, 0], 1.0
    c.w_gate.zero_(), c.w_up.zero_()
    c.w_gate[:, :, 0] = 1.0
    c.w_up[:, :, 1] = 1.0
    c.w_down.copy_(unit())
    c.forward()
    assert B.moe_get_error(c.err) == B.MOE_OK
    near(c.y, act64(v.double(), act)[0], v.double())


@pytest.mark.parametrize("act", ACTS)
def test_gradients(act):
    """u = 1 and dh = 1: dx is act'(g) with w_up zero, and act(g) with w_gate zero."""
    c = Case([len(VALUES)], W, W, act, B.MOE_SAVE_BF16)
    g = c.gate = of(c)
    c.up, c.grad_y = torch.ones_like(g), torch.ones_like(g)
    c.x.fill_(1.0)
    c.w_down.copy_(unit())
    p, dp = act64(g.double(), act)
    for w_gate, w_up, want in ((unit(), torch.zeros_like(unit()), dp), (torch.zeros_like(unit()), unit(), p)):
        c.w_gate, c.w_up = w_gate, w_up
        c.backward(weights=False)
        assert B.moe_get_error(c.err) == B.MOE_OK
        near(c.gx, want, g.double())
