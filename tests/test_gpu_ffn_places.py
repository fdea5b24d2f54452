"""Where the feed-forward block's operands may lie: rows that belong to no expert in front of the first one, results in
the places that the header allows, calls of several host threads; and a layer without tokens."""
import threading

import pytest
import torch

from combine_moe_layout_gb300 import _binding as B
from combine_moe_layout_gb300 import pipeline as P
from test_gpu_ffn import DEV, Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("counts,lead", [([5, 0, 7], 3), ([40, 90, 3], 17), ([300, 20], 200)])
def test_rows_in_front_of_the_first_expert(counts, lead):
    """The first offset is not 0: the rows before it are left as they were, and are no expert's."""
    c = Case([lead] + counts, 264, 136, save=B.MOE_SAVE_BF16, behind=2, seed=8)
    off = c.offsets[1:].contiguous()
    runs = [(e, int(off[e]), int(off[e + 1])) for e in range(len(counts))]
    for name in ("w_gate", "w_up", "w_down"):
        setattr(c, name, getattr(c, name)[1:].contiguous())
    c.offsets, c.E, c.runs = off, len(counts), lambda: runs
    c.desc = B.MoeFfnDesc(c.rows, c.H, c.I, c.E, 1, c.act, c.save, 0)
    c.x[:lead] = float("nan")
    c.forward()
    c.check_forward()
    assert bool((c.y[:lead] == 7.0).all()) and bool((c.gate[:lead] == 5).all())
    c.keep_made()
    for t in (c.grad_y, c.gate, c.up):
        t[:lead] = float("nan")
    c.backward()
    c.check_backward()
    assert bool((c.gx[:lead] == 7.0).all())


@pytest.mark.parametrize("counts,H,I", [([70, 0, 33], 264, 200), ([100], 2048, 512), ([700, 300], 512, 640)])
def test_results_in_the_inputs_places(counts, H, I):
    """h the forward's, and the rows' gradient where y's was, when no weights' gradients are wanted."""
    c = Case(counts, H, I, save=B.MOE_SAVE_BF16, seed=9)
    c.forward()
    c.grad_y = c.normal(c.rows, H)
    c.backward(weights=False)
    want = c.gx.clone()
    into = c.grad_y.clone()
    B.moe_ffn_grad(c.desc, c.offsets, c.x, c.gate, None, c.up, None, c.w_gate, c.w_up, c.w_down, into, c.h, c.gg, c.gu,
                   into, None, None, None, c.err)
    assert B.moe_get_error(c.err) == B.MOE_OK
    assert torch.equal(into, want)


def test_calls_of_several_host_threads():
    """Each with its own sizes, stream and error word."""
    cases = [Case(n, H, I, save=B.MOE_SAVE_BF16, seed=i) for i, (n, H, I) in enumerate(
        [([9], 264, 200), ([100], 2048, 512), ([300, 0, 20], 512, 392), ([40] * 70, 128, 64)])]
    for c in cases:
        c.keep_made()
    torch.cuda.synchronize()
    failed = []

    def work(c):
        try:
            with torch.cuda.device(0), torch.cuda.stream(torch.cuda.Stream()):
                c.backward()
                torch.cuda.current_stream().synchronize()
                for _ in range(20):
                    c.backward(reuse=True)
                torch.cuda.current_stream().synchronize()
        except Exception as e:  # noqa: BLE001
            failed.append(e)

    threads = [threading.Thread(target=work, args=(c,)) for c in cases]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed
    torch.cuda.synchronize()
    for c in cases:
        c.check_backward()


@pytest.mark.parametrize("save", ["bf16", "fp8"])
def test_a_layer_without_tokens(save):
    H, E, I = 64, 4, 128
    m = P.LocalMoe(0, H, E, 2, B.MoeGateOpts(B.MOE_SCORE_SOFTMAX, 1, 0, 0, 0, 0, 1.0), DEV, I)
    w = type("W", (), dict(w_gate=torch.ones((E, I, H), dtype=torch.bfloat16, device=DEV)))()
    w.w_up, w.w_down = w.w_gate, w.w_gate.reshape(E, H, I)
    x, logits = torch.empty((0, H), dtype=torch.bfloat16, device=DEV), torch.empty((0, E), device=DEV)
    out = m.forward(x, logits, w, save=save)
    gx, gl = m.backward(torch.empty_like(out), logits, w)
    assert out.shape == gx.shape == (0, H) and gl.shape == (0, E)
    assert not any(bool(t.any()) for t in (m.grad_w_gate, m.grad_w_up, m.grad_w_down))
    y, kept = m.dense(x, w.w_gate[0], w.w_up[0], w.w_down[0], save=save)
    grads = m.dense_grad(kept, x, w.w_gate[0], w.w_up[0], w.w_down[0], y)
    assert not any(bool(t.any()) for t in grads)
    v = torch.ones(H, device=DEV)
    r, n = m.norm(x, v, y, v, v)
    g = m.norm_grad(r, n, v, r, y, v, v)
    assert not any(bool(t.any()) for t in (g.w_pre, g.w_post, g.gate))
    assert m.error() == B.MOE_OK
