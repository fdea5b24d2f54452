"""Matrices of more than 2^32 elements: rows, weights and their gradients beyond what 32 bits address. Sampled rows and
experts against 64 bits, with the bars of test_gpu_ffn and test_gpu_norm."""
import pytest
import torch

from combine_moe_layout_gb300 import _binding as B
from gpu_common import require_gpu
from test_gpu_ffn import DEV, Case
from test_gpu_norm import Case as NormCase

pytestmark = pytest.mark.gpu


def needs(gb):
    require_gpu()
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < gb << 30:
        pytest.skip(f"needs {gb} GB")


@pytest.fixture(autouse=True)
def memory_given_back():
    yield
    torch.cuda.empty_cache()


def tiled(rows, n):
    """`rows` again and again, and its rows' numbers."""
    at = torch.arange(n, device=DEV) % rows.shape[0]
    return rows[at]


@pytest.mark.parametrize("save", [B.MOE_SAVE_BF16, B.MOE_SAVE_FP8])
def test_rows_beyond_2_32_elements(save):
    """One block; rows repeat with a period of 1021, which no tile shares. The short batch runs on one SM, so that its tiles
    are not shared by clusters, which add K in parts: equal rows have equal bits then."""
    needs(100)
    n, H, I, period = 640_003, 7168, 128, 1021
    small = c = Case([period], H, I, save=save, dense=True, seed=11, num_sms=1)
    small.forward()
    small.check_forward()
    small.keep_made()
    small.backward(weights=False)
    small.check_backward()
    big = Case([1], H, I, save=save, dense=True)
    big.n = big.rows = n
    big.counts = [n]
    big.desc = B.MoeFfnDesc(n, H, I, 1, 1, c.act, save, 0)
    big.w_gate, big.w_up, big.w_down = c.w_gate, c.w_up, c.w_down
    big.x = tiled(c.x, n)
    big.h, big.y = tiled(c.h, n), torch.empty_like(big.x)
    kept = [t for t in ("gate", "up", "gate_scales", "up_scales") if getattr(c, t) is not None]
    made = {t: getattr(c, t).clone() for t in kept}
    for t in kept:
        setattr(big, t, torch.empty((n, made[t].shape[1]), dtype=made[t].dtype, device=DEV))
    big.forward()
    small.forward()
    assert B.moe_get_error(big.err) == B.MOE_OK
    at = torch.arange(n, device=DEV) % period

    def check(got, want):
        for i in range(0, n, 1 << 16):
            assert torch.equal(got[i:i + (1 << 16)], want[at[i:i + (1 << 16)]]), i

    for name in ["y"] + kept:
        check(getattr(big, name), getattr(small, name))
    for t in kept:
        getattr(small, t).copy_(made[t])
        setattr(big, t, tiled(made[t], n))
    big.grad_y = tiled(small.grad_y, n)
    big.hg, big.gg, big.gu = (torch.empty((n, I), dtype=torch.bfloat16, device=DEV) for _ in range(3))
    big.gx, big.gw = big.y, [None] * 3
    big.backward(reuse=True)
    assert B.moe_get_error(big.err) == B.MOE_OK
    check(big.gx, small.gx)


def test_weights_beyond_2_32_elements():
    needs(130)
    E, H, I = 800, 4096, 1408
    counts = [(i * 7) % 5 for i in range(E)]
    counts[-1], counts[-2], counts[0] = 130, 0, 70
    c = Case([1], H, I)
    g = torch.Generator(device=DEV).manual_seed(12)
    c.counts, c.E, c.n = counts, E, sum(counts)
    c.rows = c.n
    c.save = B.MOE_SAVE_BF16
    c.desc = B.MoeFfnDesc(c.rows, H, I, E, 1, c.act, c.save, 0)
    c.offsets = torch.tensor([0] + counts, device=DEV).cumsum(0).int()
    c.x = torch.randn((c.rows, H), generator=g, device=DEV).to(torch.bfloat16)

    def weights(shape, scale):
        out = torch.empty((E, *shape), dtype=torch.bfloat16, device=DEV)
        for e in range(E):
            out[e] = torch.randn(shape, generator=g, device=DEV) * scale
        return out

    c.w_gate, c.w_up, c.w_down = weights((I, H), H ** -0.5), weights((I, H), H ** -0.5), weights((H, I), I ** -0.5)
    assert c.w_gate.numel() > 1 << 32
    c.h = torch.zeros((c.rows, I), dtype=torch.bfloat16, device=DEV)
    c.y = torch.full((c.rows, H), 7.0, dtype=torch.bfloat16, device=DEV)
    c.gate, c.up = torch.empty_like(c.h), torch.empty_like(c.h)
    runs = [r for r in Case.runs(c)]
    some = [r for r in runs if r[0] < 3 or r[0] >= E - 6 or r[0] in (371, 372, 373, 744, 745, 746)]
    c.runs = lambda: some
    c.forward()
    c.check_forward()
    c.keep_made()
    c.backward()
    c.check_backward()
    for e, a, b in runs:
        if a == b:
            assert not any(bool(t[e].any()) for t in c.gw), e


@pytest.mark.parametrize("fp32", [False, True])
def test_norms_beyond_2_32_elements(fp32):
    needs(150)
    n, H, period = 540_001, 8192, 1021
    s = NormCase(period, H, fp32, B.MOE_GATE_ROW, True, seed=13)
    s.forward()
    s.check_forward()
    s.backward()
    s.check_backward()
    b = NormCase(1, H, fp32, B.MOE_GATE_ROW, True)
    b.T, b.desc = n, B.MoeNormDesc(n, H, int(fp32), B.MOE_GATE_ROW, s.eps, s.alpha)
    b.w_pre, b.w_post = s.w_pre, s.w_post
    at = torch.arange(n, device=DEV) % period

    def check(got, want):
        for i in range(0, n, 1 << 15):
            assert torch.equal(got[i:i + (1 << 15)], want[at[i:i + (1 << 15)]]), i

    b.x, b.o, b.gate = tiled(s.x, n), tiled(s.o, n), s.gate[at]
    b.r, b.n = torch.empty_like(b.x), torch.empty((n, H), dtype=torch.bfloat16, device=DEV)
    b.forward()
    check(b.r, s.r)
    check(b.n, s.n)
    b.r = None
    b.grad_r, b.grad_n = tiled(s.grad_r, n), tiled(s.grad_n, n)
    b.gx, b.go, b.gg = b.grad_r, b.grad_n, torch.empty(n, device=DEV)  # in their places
    b.gwp, b.gw = torch.empty(H, device=DEV), torch.empty(H, device=DEV)
    work = torch.empty(B.moe_norm_workspace(b.desc), dtype=torch.uint8, device=DEV)
    B.moe_norm_grad(b.desc, b.x, b.o, b.w_post, b.gate, b.w_pre, b.grad_r, b.grad_n, b.gx, b.go, b.gwp, b.gg, b.gw, work,
                    b.err)
    assert B.moe_get_error(b.err) == B.MOE_OK
    check(b.gx, s.gx)
    check(b.go, s.go)
    check(b.gg, s.gg)
