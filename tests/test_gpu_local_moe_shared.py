"""LocalMoe.shared: results are the caller's own, and the projection runs alone where there are no adapters."""
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


@pytest.mark.parametrize("T", [1, 33, 200])
def test_the_projection_alone(T):
    """Bar: one bf16 rounding, and (K + 2) 2^-22 of the magnitudes that are added (as the projection's own tests)."""
    require_gpu()
    layer, draw = layer_and_rows(T, 128)
    x, w = draw(T, 128), draw(264, 128)
    y = layer.shared(x, w)
    assert layer.error() == B.MOE_OK
    want = x.double() @ w.double().t()
    bar = 2.0 ** -8 * want.abs() + 130 * 2.0 ** -22 * (x.double().abs() @ w.double().abs().t())
    assert bool(((y.double() - want).abs() <= bar).all())


def test_a_result_of_expert_grad_of_another_type_or_size_is_refused():
    """It goes on by address, and was read as bf16 [tokens * topk][hidden] whatever it was."""
    require_gpu()
    layer, draw = layer_and_rows(9, 128)
    x, logits = draw(9, 128), draw(9, 4).float()
    layer.route(logits)
    layer.sort(x)
    layer.packed_y.copy_(layer.packed_x)
    layer.unsort()
    for bad in (lambda px, off, gy: gy.float(), lambda px, off, gy: gy[:4], lambda px, off, gy: None):
        with pytest.raises(ValueError, match="expert_grad's result"):
            layer.backward(x, logits, bad)
    layer.backward(x, logits, lambda px, off, gy: gy)
    assert layer.error() == B.MOE_OK


@pytest.mark.parametrize("parts", [1, 2])
def test_parts_of_u(parts):
    """The bits of the entry point with as many parts; two are what shared takes by itself."""
    require_gpu()
    layer, draw = layer_and_rows(90, 128)
    x, w, la, lb = draw(90, 128), draw(264, 128), draw(3, 24, 128), draw(3, 264, 24)
    ids = (torch.arange(90) % 4 - 1).to(torch.int32).cuda()
    y = layer.shared(x, w, la, lb, None, ids, u_parts=parts)
    u, want = torch.empty((parts, 90, 24), dtype=torch.bfloat16, device="cuda:0"), torch.empty_like(y)
    B.moe_lora_linear(B.MoeLoraDesc(90, 128, 264, 24, 3, 0, parts), x, w, la, lb, None, ids, u, want, layer.err)
    assert layer.error() == B.MOE_OK and torch.equal(y, want) and layer.u.shape == (90, 24)
    if parts == 2:
        assert torch.equal(layer.shared(x, w, la, lb, None, ids), y)
