"""The norms with more rows than the CTAs' rings hold: stages are asked for again, the ring comes round several times,
and each CTA adds many rows to its columns' sums. Bars as in test_gpu_norm."""
import pytest
import torch

from combine_moe_layout_gb300 import _binding as B
from test_gpu_norm import Case

pytestmark = pytest.mark.gpu

# rows of 40: one warp, no barrier in a row; 256 to 8192: one or two vectors a thread, two to four stages; 8200 (fp32
# stream) and 12288 (bf16): four vectors a thread; 16392: straight from memory
SHAPES = [(11000, 40, False), (11000, 40, True), (11000, 256, False), (6000, 520, True), (3000, 1024, True),
          (2000, 4104, False), (2000, 7168, False), (2000, 7168, True), (2000, 8192, False), (2000, 8192, True),
          (1400, 8200, True), (1400, 12288, False), (700, 16392, True)]


@pytest.mark.parametrize("T,H,fp32", SHAPES)
@pytest.mark.parametrize("gate,post", [(B.MOE_GATE_NONE, False), (B.MOE_GATE_ROW, True), (B.MOE_GATE_CHANNEL, True)])
def test_many_rows(T, H, fp32, gate, post):
    c = Case(T, H, fp32, gate, post, seed=3)
    c.forward()
    c.check_forward()
    c.backward()
    c.check_backward()
    assert B.moe_get_error(c.err) == B.MOE_OK


@pytest.mark.parametrize("T,H,fp32", [(2000, 7168, True), (11000, 40, False), (1400, 12288, False)])
def test_many_rows_in_the_inputs_places(T, H, fp32):
    """Rows are fetched ahead while the rows before them are written: the same bits as with results beside the inputs."""
    c = Case(T, H, fp32, B.MOE_GATE_CHANNEL, True, seed=4)
    c.forward()
    c.backward()
    want = [t.clone() for t in (c.r, c.n, c.gx, c.go, c.gwp, c.gg, c.gw)]
    work = torch.empty(B.moe_norm_workspace(c.desc), dtype=torch.uint8, device=c.x.device)
    for into_o in (False, True):
        dr, dn, o = c.grad_r.clone(), c.grad_n.clone(), c.o.clone()
        go = o if into_o else dn
        B.moe_norm_grad(c.desc, c.x, o, c.w_post, c.gate, c.w_pre, dr, dn, dr, go, c.gwp, c.gg, c.gw, work, c.err)
        for got, w in zip((dr, go, c.gwp, c.gg, c.gw), want[2:]):
            assert torch.equal(got, w)
    x = c.x.clone()
    B.moe_norm(c.desc, x, c.o, c.w_post, c.gate, c.w_pre, x, c.n, c.err)
    assert torch.equal(x, want[0]) and torch.equal(c.n, want[1])
    assert B.moe_get_error(c.err) == B.MOE_OK


@pytest.mark.parametrize("fp32", [False, True])
def test_many_rows_without_a_block(fp32):
    c = Case(5000, 1000, fp32, B.MOE_GATE_NONE, False, block=False, seed=5)
    c.forward(r=None)
    c.r.copy_(c.x)
    c.check_forward()
    for with_r in (True, False):
        c.backward(with_r)
        c.check_backward(with_r)
