"""What the router and the token sort refuse on the host, without a GPU: the
checks come before any launch, so no pointer is followed."""
import ctypes

import pytest

from combine_moe_layout_gb300 import _binding as B

P = 1 << 20  # an aligned address that is never read


def call(name, desc, *args):
    """The C call; arguments that are not ctypes values are addresses."""
    a = [x if not isinstance(x, int) else ctypes.c_void_p(x or None) for x in args]
    return getattr(B.load(), name)(ctypes.byref(desc), *a, ctypes.c_void_p(None))


def desc(R=1, T=4, H=128, E=8, k=2, dtype=0, max_m=None):
    return B.MoeDesc(R, T, H, E, k, T if max_m is None else max_m, dtype, 0)


def opts(score=0, renorm=0, groups=0, keep=0, top=0, bf16=0, scale=1.0):
    return ctypes.byref(B.MoeGateOpts(score, renorm, groups, keep, top, bf16, scale))


@pytest.mark.parametrize("d,o", [
    (desc(E=1025, k=2), opts()), (desc(k=9), opts()), (desc(E=8, k=17), opts()), (desc(), opts(score=2)),
    (desc(), opts(renorm=2)), (desc(), opts(bf16=-1)), (desc(), opts(scale=float("nan"))),
    (desc(), opts(scale=float("inf"))), (desc(), opts(groups=3, keep=1, top=1)), (desc(), opts(groups=-1)),
    (desc(E=64, k=2), opts(groups=64, keep=4, top=1)), (desc(), opts(groups=4, keep=0, top=1)),
    (desc(), opts(groups=4, keep=5, top=1)), (desc(), opts(groups=4, keep=1, top=3)),
    (desc(), opts(groups=4, keep=1, top=0)), (desc(k=3), opts(groups=4, keep=1, top=1)),
])
def test_gate_refuses(d, o):
    assert call("moe_gate", d, o, P, 0, P, P, P) == B.MOE_EINVAL
    assert call("moe_gate_grad", d, o, P, P, P, P, P) == B.MOE_EINVAL


@pytest.mark.parametrize("bad", [(0, 0, P, P, P), (P, 0, 0, P, P), (P, 0, P, 0, P), (P, 0, P, P, 0),
                                 (P + 2, 0, P, P, P), (P, P + 2, P, P, P), (P, 0, P + 1, P, P), (P, 0, P, P + 2, P),
                                 (P, 0, P, P, P + 1)])
def test_gate_refuses_missing_or_unaligned_buffers(bad):
    assert call("moe_gate", desc(), opts(), *bad) == B.MOE_EINVAL


@pytest.mark.parametrize("bad", [(0, P, P, P, P), (P, 0, P, P, P), (P, P, 0, P, P), (P, P, P, 0, P), (P, P, P, P, 0),
                                 (P + 2, P, P, P, P), (P, P, P, P + 2, P)])
def test_gate_grad_refuses_missing_or_unaligned_buffers(bad):
    assert call("moe_gate_grad", desc(), opts(), *bad) == B.MOE_EINVAL
    assert call("moe_gate_grad", desc(), opts(bf16=1), P + 1, P, P, P, P) == B.MOE_EINVAL


def test_null_descriptors_are_refused():
    lib = B.load()
    v = ctypes.c_void_p(P)
    assert lib.moe_gate(None, opts(), v, None, v, v, v, None) == B.MOE_EINVAL
    assert lib.moe_gate(ctypes.byref(desc()), None, v, None, v, v, v, None) == B.MOE_EINVAL
    assert lib.moe_sort(None, v, v, None, v, v, None, v, v, None) == B.MOE_EINVAL


SORT = [P, P, 0, P, P, 0, P, P]  # idx, x, scales, offsets, packed, packed scales, tok, err


@pytest.mark.parametrize("at,value", [(0, 0), (1, 0), (3, 0), (4, 0), (6, 0), (7, 0), (0, P + 2), (1, P + 8), (3, P + 2),
                                      (4, P + 8), (6, P + 1), (7, P + 2)])
def test_sort_refuses_missing_or_unaligned_buffers(at, value):
    args = list(SORT)
    args[at] = value
    assert call("moe_sort", desc(), *args) == B.MOE_EINVAL


@pytest.mark.parametrize("d", [desc(T=5, max_m=4), desc(H=4), desc(H=192, dtype=1), desc(H=192, dtype=2), desc(E=8193, k=1),
                               desc(R=3), desc(dtype=3), desc(T=-1)])
def test_sort_refuses_sizes(d):
    args = list(SORT)
    args[2] = args[5] = P
    assert call("moe_sort", d, *args) == B.MOE_EINVAL


@pytest.mark.parametrize("dtype,scales,packed_scales", [(1, 0, P), (1, P, 0), (1, P + 2, P), (1, P, P + 1), (2, 0, 0)])
def test_sort_of_fp8_rows_wants_scales(dtype, scales, packed_scales):
    args = list(SORT)
    args[2], args[5] = scales, packed_scales
    assert call("moe_sort", desc(dtype=dtype), *args) == B.MOE_EINVAL


@pytest.mark.parametrize("name,good", [("moe_sort_grad", [P] * 4), ("moe_unsort", [P] * 5), ("moe_unsort_grad", [P] * 7)])
def test_the_other_calls_refuse_missing_or_unaligned_buffers(name, good):
    for at in range(len(good)):
        for value in (0, P + 2):
            args = list(good)
            args[at] = value
            if name == "moe_unsort_grad" and at == 5 and value == 0:
                continue  # grad_weights is optional
            assert call(name, desc(), *args) == B.MOE_EINVAL, (name, at, value)


def test_the_binding_refuses_host_and_strided_tensors():
    import torch
    d, o = desc(), B.MoeGateOpts(0, 0, 0, 0, 0, 0, 1.0)
    host = torch.zeros((4, 8))
    with pytest.raises(ValueError):
        B.moe_gate(d, o, host, None, host, host, host)


def lora_desc(T=4, K=64, N=64, r=16, A=2, sms=0):
    return B.MoeLoraDesc(T, K, N, r, A, sms)


LORA = [P] * 9  # x, w, lora_a, lora_b, scales, adapter, u, y, err


@pytest.mark.parametrize("d", [lora_desc(T=-1), lora_desc(K=60), lora_desc(K=0), lora_desc(N=12), lora_desc(N=0),
                               lora_desc(r=12), lora_desc(r=0), lora_desc(r=264), lora_desc(A=-1), lora_desc(sms=-1),
                               lora_desc(A=1 << 26, N=64)])
def test_lora_refuses_sizes(d):
    assert call("moe_lora_linear", d, *LORA) == B.MOE_EINVAL


@pytest.mark.parametrize("at,value", [(0, 0), (1, 0), (2, 0), (3, 0), (5, 0), (6, 0), (7, 0), (8, 0), (0, P + 8), (1, P + 2),
                                      (2, P + 8), (3, P + 8), (4, P + 2), (5, P + 2), (6, P + 8), (7, P + 8),
                                      (8, P + 2)])
def test_lora_refuses_missing_or_unaligned_buffers(at, value):
    args = list(LORA)
    args[at] = value
    assert call("moe_lora_linear", lora_desc(), *args) == B.MOE_EINVAL


def test_lora_with_no_tokens_does_nothing():
    assert call("moe_lora_linear", lora_desc(T=0), 0, 0, 0, 0, 0, 0, 0, 0, P) == B.MOE_OK
