"""What pipeline.LocalMoe refuses, without a GPU: sizes and types are compared before any call, so that a wrong one is
an error instead of a read out of range. (Tensors in host memory that pass are refused by the binding.)"""
import pytest
import torch

from combine_moe_layout_gb300 import _binding as B
from combine_moe_layout_gb300 import pipeline as P

T, H, E, K = 6, 16, 4, 2


def layer(bf16=0, inter=0):
    return P.LocalMoe(T, H, E, K, B.MoeGateOpts(0, 1, 0, 0, 0, bf16, 1.0), "cpu", inter)


def z(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


def f(*shape):
    return z(*shape, dtype=torch.float32)


def refused(name, call, *args, **kw):
    with pytest.raises(ValueError, match=rf"LocalMoe: {name} "):
        call(*args, **kw)


@pytest.mark.parametrize("logits", [f(T, E + 1), f(T - 1, E), z(T, E), f(T * E)])
def test_route_refuses_logits(logits):
    refused("logits", layer().route, logits)


def test_route_goes_by_the_type_of_the_options():
    refused("logits", layer(bf16=1).route, f(T, E))
    refused("bias", layer().route, f(T, E), f(E - 1))
    refused("bias", layer().route, f(T, E), z(E))


@pytest.mark.parametrize("x", [z(T, H + 8), z(T + 1, H), f(T, H)])
def test_sort_refuses_rows(x):
    refused("x", layer().sort, x)


@pytest.mark.parametrize("field,bad", [("w_gate", z(E, 128, H - 8)), ("w_up", z(E - 1, 128, H)), ("w_down", z(E, H, 64)),
                                       ("w_gate", f(E, 128, H))])
def test_experts_refuse_weights(field, bad):
    class W:
        w_gate, w_up, w_down = z(E, 128, H), z(E, 128, H), z(E, H, 128)

    w = W()
    setattr(w, field, bad)
    refused(field, layer(inter=128).experts, w)


def test_experts_of_a_layer_without_a_width_are_refused():
    with pytest.raises(ValueError, match="inter"):
        layer().experts(None)


@pytest.mark.parametrize("name,grad_out,logits", [("grad_out", z(T, H - 8), f(T, E)), ("grad_out", f(T, H), f(T, E)),
                                                  ("logits", z(T, H), f(T, E - 1))])
def test_backward_refuses(name, grad_out, logits):
    refused(name, layer().backward, grad_out, logits, lambda px, off, gy: gy)


GOOD = dict(x=z(5, H), w=z(24, H), lora_a=z(3, 8, H), lora_b=z(3, 24, 8), scales=f(3), adapter=z(5, dtype=torch.int32))


@pytest.mark.parametrize("name,bad", [
    ("x", f(5, H)), ("x", z(5 * H)), ("w", z(24, H + 8)), ("w", f(24, H)), ("lora_a", z(3, 8, H - 8)), ("lora_a", z(3, 8)),
    ("lora_b", z(2, 24, 8)), ("lora_b", z(3, 16, 8)), ("lora_b", z(3, 24, 16)), ("scales", f(2)), ("scales", z(3)),
    ("adapter", z(4, dtype=torch.int32)), ("adapter", z(5, dtype=torch.int64)), ("lora_b", None), ("adapter", None),
])
def test_shared_refuses(name, bad):
    refused(name, layer().shared, **{**GOOD, name: bad})


def test_shared_without_adapters_takes_none_of_their_arguments():
    refused("adapter", layer().shared, GOOD["x"], GOOD["w"], adapter=GOOD["adapter"])


@pytest.mark.parametrize("parts", [0, 3, None])
def test_shared_refuses_parts(parts):
    refused("u_parts", layer().shared, **GOOD, u_parts=parts)


def test_what_passes_reaches_the_binding():
    w = type("W", (), dict(w_gate=z(E, 128, H), w_up=z(E, 128, H), w_down=z(E, H, 128)))()
    for call in (lambda: layer().route(f(T, E), f(E)), lambda: layer().route(f(2, 3, E)),
                 lambda: layer().sort(z(1, T, H)), lambda: layer(bf16=1).route(z(T, E)), lambda: layer().sort(z(T, H)),
                 lambda: layer(inter=128).experts(w), lambda: layer().shared(**GOOD),
                 lambda: layer().shared(GOOD["x"], GOOD["w"]), lambda: layer().backward(z(T, H), f(T, E), None)):
        with pytest.raises(ValueError, match="libmoe_layout takes device tensors"):
            call()


@pytest.mark.parametrize("save", ["fp16", 1, "none"])
def test_what_is_kept_is_refused(save):
    w = type("W", (), dict(w_gate=z(E, 128, H), w_up=z(E, 128, H), w_down=z(E, H, 128)))()
    refused("save", layer(inter=128).experts, w, save=save)
    refused("save", layer().dense, z(5, H), z(24, H), z(24, H), z(H, 24), save=save)


def test_backward_with_weights_follows_a_forward_that_kept():
    w = type("W", (), dict(w_gate=z(E, 128, H), w_up=z(E, 128, H), w_down=z(E, H, 128)))()
    with pytest.raises(ValueError, match="follows a forward with save"):
        layer(inter=128).backward(z(T, H), f(T, E), w)
    w.w_up = z(E, 128, H + 8)
    refused("w_up", layer(inter=128).backward, z(T, H), f(T, E), w)


DENSE = dict(x=z(5, H), w_gate=z(24, H), w_up=z(24, H), w_down=z(H, 24))


@pytest.mark.parametrize("name,bad", [("x", f(5, H)), ("x", z(5 * H)), ("w_gate", z(24, H + 8)), ("w_up", z(16, H)),
                                      ("w_down", z(24, H)), ("w_down", f(H, 24))])
def test_dense_refuses(name, bad):
    refused(name, layer().dense, **{**DENSE, name: bad})


@pytest.mark.parametrize("name,bad", [("x", z(4, H)), ("w_gate", z(16, H)), ("w_up", f(24, H)), ("w_down", z(24, H)),
                                      ("grad_y", z(5, H + 8))])
def test_dense_grad_refuses(name, bad):
    kept = P.KeptFfn(B.MoeFfnDesc(5, H, 24, 1, 1, 0, 1, 0), z(5, 24), z(5, 24), None, None)
    refused(name, layer().dense_grad, kept, **{**DENSE, "grad_y": z(5, H), name: bad})


NORM = dict(x=z(5, H), w_pre=f(H), o=z(5, H), w_post=f(H), gate=f(H))


@pytest.mark.parametrize("name,bad", [("x", z(5 * H)), ("x", z(5, H, dtype=torch.float16)), ("w_pre", z(H)),
                                      ("w_pre", f(H + 8)), ("o", f(5, H)), ("o", z(4, H)), ("w_post", z(H)),
                                      ("w_post", f(5)), ("gate", f(5)), ("gate", z(H)), ("by", "rows")])
def test_norm_refuses(name, bad):
    refused(name, layer().norm, **{**NORM, name: bad})
    if name != "x":
        good = {("r" if k == "x" else k): v for k, v in NORM.items()}
        refused(name, layer().norm_grad, **{**good, "grad_n": z(5, H), name: bad})


def test_norm_without_a_block_takes_nothing_of_it():
    refused("w_post or gate", layer().norm, z(5, H), f(H), gate=f(H))
    refused("grad_r", layer().norm_grad, z(5, H), z(5, H), f(H), f(5, H))
    refused("grad_n", layer().norm_grad, z(5, H), f(5, H), f(H))


def test_what_passes_of_training_reaches_the_binding():
    w = type("W", (), dict(w_gate=z(E, 128, H), w_up=z(E, 128, H), w_down=z(E, H, 128)))()
    kept = P.KeptFfn(B.MoeFfnDesc(5, H, 24, 1, 1, 0, 1, 0), z(5, 24), z(5, 24), None, None)
    for call in (lambda: layer(inter=128).experts(w, save="bf16"), lambda: layer(inter=128).experts(w, save="fp8"),
                 lambda: layer().dense(**DENSE), lambda: layer().dense(**DENSE, save="bf16"),
                 lambda: layer().dense_grad(kept, **DENSE, grad_y=z(5, H)), lambda: layer().norm(**NORM),
                 lambda: layer().norm(f(5, H), f(H)), lambda: layer().norm(**{**NORM, "gate": f(5)}, by="row"),
                 lambda: layer().norm_grad(f(5, H), z(5, H), f(H), f(5, H))):
        with pytest.raises(ValueError, match="libmoe_layout takes device tensors"):
            call()
