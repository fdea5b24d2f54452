"""Shapes at the border between a CTA for each 128-wide tile and CTAs that walk 256-wide ones, called again and again
back to back behind one another: the same bits every time, within the projection's bar."""
from __future__ import annotations

import pytest
import torch

from combine_moe_layout_gb300 import _binding as B
from test_gpu_lora import check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,K,N,r,A", [
    (1024, 512, 2432, 16, 4),   # 8 x 19 = 152 tiles of 128
    (1156, 520, 1920, 24, 3),   # 10 x 15 of 128, the last ending inside a warp
    (1156, 520, 2048, 24, 3),   # 160 of 128, 80 of 256
    (2500, 520, 2048, 24, 6),   # 160 of 256: CTAs walk
    (300, 264, 6400, 72, 5),    # u in two blocks of 64 columns
])
def test_again_and_again(T, K, N, r, A):
    x, w, la, lb, sc, ids, want = check(T, K, N, r, A, "runs")
    d = B.MoeLoraDesc(T, K, N, r, A, 0)
    u = torch.empty((T, r), dtype=torch.bfloat16, device="cuda:0")
    ys = [torch.empty((T, N), dtype=torch.bfloat16, device="cuda:0") for _ in range(3)]
    err = torch.zeros(1, dtype=torch.int32, device="cuda:0")
    for i in range(60):
        B.moe_lora_linear(d, x, w, la, lb, sc, ids, u, ys[i % 3], err)
    assert B.moe_get_error(err) == B.MOE_OK and all(torch.equal(y, want) for y in ys)
