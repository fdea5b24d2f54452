"""A captured training step of the one-device layer beside eager steps that keep another format."""
from __future__ import annotations

import pytest
import torch

from combine_moe_layout_gb300 import _binding as B
from test_gpu_local_moe_training import Step

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("first,other", [("fp8", "bf16"), ("bf16", "fp8")])
def test_a_graph_outlives_a_forward_with_another_format(first, other):
    """Captured after an eager step, so that the kept buffers are the ordinary pool's; then a step that keeps the other
    format, and tensors that would take the place of buffers given up. Every replay has the captured step's results and
    leaves those tensors alone."""
    s = Step(T=70)
    want = {k: v.clone() for k, v in s.backward(s.forward(first)[0]).items()}
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = s.backward(s.forward(first)[0])
    s.backward(s.forward(other)[0])
    room = [torch.full((s.layer.packed_x.shape[0], s.I), 3.0, dtype=torch.bfloat16, device="cuda") for _ in range(16)]
    room += [torch.full((s.layer.packed_x.shape[0], s.I), 3, dtype=torch.uint8, device="cuda") for _ in range(16)]
    for _ in range(2):
        g.replay()
        torch.cuda.synchronize()
        for name, w in want.items():
            assert torch.equal(got[name], w), name
        assert all(bool((t == 3).all()) for t in room)
        s.backward(s.forward(other)[0])
    assert s.layer.error() == B.MOE_OK


@pytest.mark.parametrize("save", ["fp8", "bf16"])
def test_a_first_step_in_a_capture(save):
    """What the layer keeps and the gradients' buffers are allocated in the capture, and used outside of it too, also
    when the graph is gone."""
    s, ref = Step(T=70), Step(T=70)
    want = {k: v.clone() for k, v in ref.backward(ref.forward(save)[0]).items()}
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = s.backward(s.forward(save)[0])
    for _ in range(2):
        g.replay()
        torch.cuda.synchronize()
        for name, w in want.items():
            assert torch.equal(got[name], w), name
        eager = s.backward(s.forward(save)[0])
        for name, w in want.items():
            assert torch.equal(eager[name], w), name
    torch.cuda.synchronize()
    del g, got
    torch.cuda.empty_cache()
    room = [torch.full((1 << 20,), 3, dtype=torch.uint8, device="cuda") for _ in range(32)]
    eager = s.backward(s.forward(save)[0])
    for name, w in want.items():
        assert torch.equal(eager[name], w), name
    assert all(bool((t == 3).all()) for t in room)
    assert s.layer.error() == B.MOE_OK
