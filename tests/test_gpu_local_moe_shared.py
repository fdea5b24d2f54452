"""LocalMoe.shared: results are the caller's own."""
from __future__ import annotations

import pytest
import torch

from combine_moe_layout_gb300 import _binding as B
from combine_moe_layout_gb300 import pipeline as P
from gpu_common import require_gpu

pytestmark = pytest.mark.gpu


def layer_and_rows(T, K):
    g = torch.Generator().manual_seed(1)
    layer = P.LocalMoe(T, K, 4, 1, B.MoeGateOpts(B.MOE_SCORE_SOFTMAX, 1, 0, 0, 0, 0, 1.0), "cuda:0")

    def draw(*shape):
        return torch.randn(shape, generator=g).to(torch.bfloat16).cuda()

    return layer, draw


def test_a_result_stays_when_another_projection_of_its_shape_follows():
    """A shared expert's gate and up projections: the same sizes, other weights."""
    require_gpu()
    layer, draw = layer_and_rows(33, 128)
    x, ids = draw(33, 128), (torch.arange(33) % 3 - 1).to(torch.int32).cuda()
    la, lb = draw(2, 16, 128), draw(2, 256, 16)
    gate = layer.shared(x, draw(256, 128), la, lb, None, ids)
    kept = gate.clone()
    up = layer.shared(x, draw(256, 128), la, lb, None, ids)
    assert layer.error() == B.MOE_OK
    assert torch.equal(gate, kept) and not torch.equal(gate, up)
