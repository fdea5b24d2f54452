"""LocalMoe on streams other than the current one, each call beside work that another stream still has to do.

The expected values are the same calls' on the current stream with nothing else running; every kernel gives the same
bits each time, so results have to be equal."""
from __future__ import annotations

import pytest
import torch

from combine_moe_layout_gb300 import _binding as B
from combine_moe_layout_gb300 import pipeline as P
from gpu_common import require_gpu

pytestmark = pytest.mark.gpu
T, H, E, K = 70, 264, 12, 3
BUSY = 100_000_000  # cycles: 50 ms or more


def opts():
    return B.MoeGateOpts(B.MOE_SCORE_SOFTMAX, 1, 0, 0, 0, 0, 1.0)


def data():
    g = torch.Generator().manual_seed(2)
    x = torch.randn((T, H), generator=g).to(torch.bfloat16).cuda()
    go = torch.randn((T, H), generator=g).to(torch.bfloat16).cuda()
    return x, torch.randn((T, E), generator=g).cuda(), go


def forward(layer, x, logits, stream=None):
    layer.route(logits, stream=stream)
    layer.sort(x, stream=stream)


def twice(px, off, gy):
    return gy * 2


def expected():
    x, logits, go = data()
    layer = P.LocalMoe(T, H, E, K, opts(), "cuda:0")
    forward(layer, x, logits)
    layer.packed_y.copy_(layer.packed_x)
    layer.unsort()
    gx, gl = layer.backward(go, logits, twice)
    torch.cuda.synchronize()
    return x, logits, go, layer, gx.clone(), gl.clone()


@pytest.mark.parametrize("busy", ["current", "side"])
def test_first_backward_on_a_side_stream(busy):
    """The gradients' buffers are made, and expert_grad runs, in the order of the call's own stream."""
    require_gpu()
    x, logits, go, ref, gx_ref, gl_ref = expected()
    layer = P.LocalMoe(T, H, E, K, opts(), "cuda:0")
    forward(layer, x, logits)
    layer.packed_y.copy_(layer.packed_x)
    layer.unsort()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side if busy == "side" else torch.cuda.current_stream()):
        torch.cuda._sleep(BUSY)
    gx, gl = layer.backward(go, logits, twice, stream=side)
    side.synchronize()
    torch.cuda.synchronize()
    assert layer.error() == B.MOE_OK
    assert torch.equal(layer.grad_y, ref.grad_y) and torch.equal(layer.grad_weights, ref.grad_weights)
    assert torch.equal(gx, gx_ref) and torch.equal(gl, gl_ref)


@pytest.mark.parametrize("given", [True, False])
def test_a_layer_made_behind_other_work(given):
    """A layer's buffers are ready on another stream, given or current, only after what the stream that made them did
    before: here the error word is cleared behind a sleep, and the call latches an error on the other stream."""
    require_gpu()
    _, logits, _ = data()
    logits[3, 4] = float("nan")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(BUSY)
    layer = P.LocalMoe(T, H, E, K, opts(), "cuda:0")
    if given:
        layer.route(logits, stream=side)
    else:
        with torch.cuda.stream(side):
            layer.route(logits)
    torch.cuda.synchronize()
    assert layer.error(side) == B.MOE_EINVAL


def test_memory_of_a_dropped_layer_is_not_given_out_while_its_stream_works():
    require_gpu()
    x, logits, _ = data()
    layer = P.LocalMoe(T, H, E, K, opts(), "cuda:0")
    forward(layer, x, logits)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(BUSY)
    layer.sort(x, stream=side)
    shape, at = layer.packed_x.shape, layer.packed_x.data_ptr()
    del layer
    other = [torch.full(shape, 7.0, dtype=torch.bfloat16, device="cuda:0") for _ in range(4)]
    assert all(o.data_ptr() != at for o in other)
    torch.cuda.synchronize()
    assert all(bool((o == 7.0).all()) for o in other)


def projection(N, r, seed):
    g = torch.Generator().manual_seed(seed)

    def draw(*shape):
        return torch.randn(shape, generator=g).to(torch.bfloat16).cuda()

    return draw(N, H), draw(3, r, H), draw(3, N, r)


def test_shared_of_two_shapes_on_a_side_stream():
    """What the first projection still writes on the side stream is not given out to the current one."""
    require_gpu()
    x, _, _ = data()
    ids = (torch.arange(T) % 4 - 1).to(torch.int32).cuda()
    layer = P.LocalMoe(T, H, E, K, opts(), "cuda:0")
    first, second = projection(512, 16, 5), projection(264, 8, 6)
    want = [layer.shared(x, *p, None, ids).clone() for p in (first, second)]
    layer = P.LocalMoe(T, H, E, K, opts(), "cuda:0")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(BUSY)
    y = layer.shared(x, *first, None, ids, stream=side)
    shape = y.shape
    del y
    got = layer.shared(x, *second, None, ids, stream=side)
    other = [torch.full(shape, 7.0, dtype=torch.bfloat16, device="cuda:0") for _ in range(4)]
    torch.cuda.synchronize()
    assert layer.error() == B.MOE_OK and torch.equal(got, want[1])
    assert all(bool((o == 7.0).all()) for o in other)


def test_shared_on_two_streams_at_a_time():
    require_gpu()
    x, _, _ = data()
    ids = (torch.arange(T) % 4 - 1).to(torch.int32).cuda()
    layer = P.LocalMoe(T, H, E, K, opts(), "cuda:0")
    ps = [projection(512, 16, 5), projection(512, 16, 6)]
    want = [layer.shared(x, *p, None, ids).clone() for p in ps]
    sides = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    with torch.cuda.stream(sides[0]):
        torch.cuda._sleep(BUSY)
    got = [layer.shared(x, *p, None, ids, stream=s) for p, s in zip(ps, sides)]
    torch.cuda.synchronize()
    assert layer.error() == B.MOE_OK
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_a_captured_layer_replays():
    """Forward and backward captured together, on a stream that did not make the layer, and replayed on new inputs."""
    require_gpu()
    x, logits, go, ref, gx_ref, gl_ref = expected()
    layer = P.LocalMoe(T, H, E, K, opts(), "cuda:0")
    xs, ls = torch.zeros_like(x), torch.zeros_like(logits)

    def step():
        forward(layer, xs, ls)
        layer.packed_y.copy_(layer.packed_x)
        layer.unsort()
        return layer.backward(go, ls, twice)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gx, gl = step()
    xs.copy_(x)
    ls.copy_(logits)
    graph.replay()
    torch.cuda.synchronize()
    assert layer.error() == B.MOE_OK
    assert torch.equal(gx, gx_ref) and torch.equal(gl, gl_ref)


def test_a_layer_made_in_a_capture():
    """Its buffers are the graph's; calls after the capture use them too."""
    require_gpu()
    _, logits, _ = data()
    ref = P.LocalMoe(T, H, E, K, opts(), "cuda:0")
    ref.route(logits)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer = P.LocalMoe(T, H, E, K, opts(), "cuda:0")
        layer.route(logits)
    graph.replay()
    assert layer.error() == B.MOE_OK and torch.equal(layer.topk_idx, ref.topk_idx)
    layer.topk_idx.zero_()
    layer.route(logits)
    assert layer.error() == B.MOE_OK and torch.equal(layer.topk_idx, ref.topk_idx)
