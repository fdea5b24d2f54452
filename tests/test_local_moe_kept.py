"""What pipeline.LocalMoe keeps of a forward for its backward, on the host alone: the binding's calls are stubs that
note their names, so that what a sequence of calls would launch can be read."""
import pytest
import torch

from combine_moe_layout_gb300 import _binding as B
from combine_moe_layout_gb300 import pipeline as P

T, H, E, K, I = 6, 16, 4, 2, 128


def z(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


X, LOGITS = z(T, H), z(T, E, dtype=torch.float32)


class Weights:
    def __init__(self):
        self.w_gate, self.w_up, self.w_down = z(E, I, H), z(E, I, H), z(E, H, I)


@pytest.fixture
def calls(monkeypatch):
    """The names of the library's calls, in order; no kernel runs."""
    names = []
    for name in ("moe_gate", "moe_sort", "moe_ffn", "moe_expert_gate_up", "moe_expert_down", "moe_unsort",
                 "moe_unsort_grad", "moe_ffn_grad", "moe_sort_grad", "moe_gate_grad"):
        monkeypatch.setattr(B, name, lambda *a, _name=name, **k: names.append(_name))
    return names


def layer():
    return P.LocalMoe(T, H, E, K, B.MoeGateOpts(0, 1, 0, 0, 0, 0, 1.0), "cpu", I)


def refused_backward(m, calls):
    calls.clear()
    with pytest.raises(ValueError, match="follows a forward with save"):
        m.backward(X, LOGITS, Weights())
    assert calls == []


def test_backward_follows_a_forward_that_kept(calls):
    m = layer()
    m.forward(X, LOGITS, Weights(), save="bf16")
    calls.clear()
    m.backward(X, LOGITS, Weights())
    m.backward(X, LOGITS, Weights())  # and again: it leaves what was kept as it is
    assert calls == ["moe_unsort_grad", "moe_ffn_grad", "moe_sort_grad", "moe_gate_grad"] * 2


@pytest.mark.parametrize("then", ["route", "sort", "experts"])
def test_another_batch_in_the_layer_ends_what_was_kept(calls, then):
    """topk_idx and the weights, the rows and their offsets, and the rows' outputs are the next batch's then."""
    m = layer()
    m.forward(X, LOGITS, Weights(), save="bf16")
    {"route": lambda: m.route(LOGITS), "sort": lambda: m.sort(X), "experts": lambda: m.experts(Weights())}[then]()
    refused_backward(m, calls)


@pytest.mark.parametrize("bad", [dict(save="fp16"), dict(x=z(T, H + 8)), dict(bias=z(E)),
                                 dict(logits=z(T, E + 1, dtype=torch.float32)), dict(w_up=z(E, I, H + 8))])
def test_a_refused_forward_changes_nothing(calls, bad):
    """It is refused before its first launch, and the batch before it can still be taken back."""
    m, w = layer(), Weights()
    m.forward(X, LOGITS, w, save="bf16")
    calls.clear()
    b = Weights()
    b.w_up = bad.get("w_up", b.w_up)
    with pytest.raises(ValueError, match="LocalMoe"):
        m.forward(bad.get("x", X), bad.get("logits", LOGITS), b, bad.get("bias"), save=bad.get("save", "bf16"))
    assert calls == []
    m.backward(X, LOGITS, w)
    assert "moe_ffn_grad" in calls


@pytest.mark.parametrize("failing", ["moe_gate", "moe_sort", "moe_ffn"])
def test_a_call_that_fails_on_its_way_leaves_nothing_kept(calls, monkeypatch, failing):
    m = layer()
    m.forward(X, LOGITS, Weights(), save="bf16")

    def fail(*args, **kw):
        raise B.MoeError(B.MOE_ECUDA, failing)

    monkeypatch.setattr(B, failing, fail)
    with pytest.raises(B.MoeError):
        m.forward(X, LOGITS, Weights(), save="bf16")
    refused_backward(m, calls)


def test_each_format_keeps_its_buffers(calls):
    """A captured forward writes to the addresses of its capture at every replay, whatever a call between them kept."""
    m = layer()
    held = {}
    for save in ("fp8", "bf16", "fp8", "bf16"):
        m.forward(X, LOGITS, Weights(), save=save)
        assert m.kept.desc.save == P.SAVE[save]
        now = [t.data_ptr() for t in (m.kept.gate, m.kept.up, m.kept.gate_scales, m.kept.up_scales) if t is not None]
        assert held.setdefault(save, (m.kept, now)) == (m.kept, now)
        m.forward(X, LOGITS, Weights())  # nor one that keeps nothing
    assert len({p for _, now in held.values() for p in now}) == 6


def test_every_formats_buffers_stay_for_a_stream(calls, monkeypatch):
    """They are given out again, after the layer, only when every stream that used it has passed them."""
    m = layer()
    for save in ("fp8", "bf16"):
        m.forward(X, LOGITS, Weights(), save=save)
    seen = []
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: seen.append(t.data_ptr()))
    m._keep_for([None])
    for k in m._kept_by.values():
        for t in (k.gate, k.up, k.gate_scales, k.up_scales):
            assert t is None or t.data_ptr() in seen


class Experts(torch.nn.Module):
    """The caller's own experts, which hold their weights and give their gradient when they are called."""

    def __init__(self):
        super().__init__()
        self.w_gate, self.w_up, self.w_down = (torch.nn.Parameter(t) for t in vars(Weights()).values())
        self.asked = 0

    def forward(self, packed_x, region_offsets, grad_y):
        self.asked += 1
        return grad_y


@pytest.mark.parametrize("save", [None, "bf16"])
def test_what_can_be_called_is_called_whatever_it_holds(calls, save):
    m, own = layer(), Experts()
    m.forward(X, LOGITS, Weights(), save=save)
    calls.clear()
    m.backward(X, LOGITS, own)
    assert own.asked == 1 and calls == ["moe_unsort_grad", "moe_sort_grad", "moe_gate_grad"]
    assert m.grad_w_gate is None
