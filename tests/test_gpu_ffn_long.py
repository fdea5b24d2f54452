"""Weights' gradients over more rows than a tile can multiply in the time that a wait for one copy may take."""
import pytest
import torch

from combine_moe_layout_gb300 import _binding as B
from gpu_common import require_gpu

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def test_sums_over_2_27_rows():
    """Widths of 8 (2 GB a matrix), two million K blocks to a tile, of which there are three. All rows but a few are
    zero, and those of the few hold one power of two each, at ends of blocks and beyond 2^31 bytes of the matrices, so
    that every sum is exact: act(g) u = 0 for g = 0 with u anything, act'(0) = 1/2."""
    require_gpu()
    n, W = (1 << 27) + 5, 8
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB")
    x, dy, gate, up, h, gg, gu, gx = (torch.zeros((n, W), dtype=torch.bfloat16, device=DEV) for _ in range(8))
    rows = [0, 63, 64, (1 << 26) + 17, n - 6, n - 1]
    eye = torch.eye(W, dtype=torch.bfloat16, device=DEV)[None].contiguous()
    for k, r in enumerate(rows):
        x[r], dy[r], up[r] = 2.0 ** k, 1.0, 4.0
    gws = [torch.full((1, W, W), 9.0, dtype=torch.bfloat16, device=DEV) for _ in range(3)]
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    desc = B.MoeFfnDesc(n, W, W, 1, 1, B.MOE_ACT_SILU, B.MOE_SAVE_BF16, 0)
    B.moe_ffn_grad(desc, None, x, gate, None, up, None, eye, eye, eye, dy, h, gg, gu, gx, *gws, err)
    assert B.moe_get_error(err) == B.MOE_OK
    # dh = 1 in the few rows, dg = dh u / 2 = 2, du = 0: dw_gate = sum 2 x = 2 (2^6 - 1) in every place
    assert bool((gws[0] == 2.0 * (2 ** len(rows) - 1)).all())
    assert not gws[1].any() and not gws[2].any()
    want = torch.zeros(n, dtype=torch.bfloat16, device=DEV)
    want[rows] = 2.0
    assert bool((gx == want[:, None]).all())


def test_whole_blocks_before_the_first_tail():
    """Only the last expert has rows behind its last whole K block: whoever clears them waits through all the others."""
    require_gpu()
    from test_gpu_ffn import Case

    c = Case([64 * 30] * 20 + [33], 264, 200, save=B.MOE_SAVE_BF16, behind=2, seed=9, num_sms=3)
    c.keep_made()
    c.backward()
    c.check_backward()
