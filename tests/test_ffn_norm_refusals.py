"""What the feed-forward block and the norms refuse on the host, without a GPU: the checks come before any launch, so
no pointer is followed."""
import ctypes

import pytest

from combine_moe_layout_gb300 import _binding as B

P = 1 << 20  # an aligned address that is never read


def call(name, desc, args):
    a = [ctypes.c_void_p(x or None) for x in args]
    return getattr(B.load(), name)(ctypes.byref(desc), *a, ctypes.c_void_p(None))


def ffn(rows=4, H=128, I=128, E=2, R=1, act=0, save=1, sms=0):
    return B.MoeFfnDesc(rows, H, I, E, R, act, save, sms)


FFN = [P] * 12        # offsets, x, 3 weights, h, y, gate, scales, up, scales, err
FFN_GRAD = [P] * 18   # offsets, x, gate, scales, up, scales, 3 weights, grad_y, h, grad_gate, grad_up, grad_x, 3, err
SIZES = [ffn(rows=-1), ffn(H=0), ffn(H=12), ffn(I=4), ffn(I=130), ffn(E=0), ffn(E=2049),
         ffn(R=0), ffn(act=2), ffn(act=-1), ffn(save=3), ffn(save=2, I=192), ffn(sms=-1), ffn(E=2048, R=1 << 21),
         ffn(E=2048, H=1 << 18, I=1 << 18)]


@pytest.mark.parametrize("d", SIZES)
def test_ffn_refuses_sizes(d):
    assert call("moe_ffn", d, FFN) == B.MOE_EINVAL
    assert call("moe_ffn_grad", d, FFN_GRAD) == B.MOE_EINVAL


@pytest.mark.parametrize("at", range(12))
@pytest.mark.parametrize("value", [0, P + 2])
def test_ffn_refuses_missing_or_unaligned_buffers(at, value):
    args = list(FFN)
    args[at] = value
    assert call("moe_ffn", ffn(save=2), args) == B.MOE_EINVAL


@pytest.mark.parametrize("at", range(18))
@pytest.mark.parametrize("value", [0, P + 2])
def test_ffn_grad_refuses_missing_or_unaligned_buffers(at, value):
    args = list(FFN_GRAD)
    args[at] = value
    assert call("moe_ffn_grad", ffn(save=2), args) == B.MOE_EINVAL


def test_ffn_grad_needs_something_kept():
    assert call("moe_ffn_grad", ffn(save=0), FFN_GRAD) == B.MOE_EINVAL


def test_ffn_without_rows_is_nothing():
    assert call("moe_ffn", ffn(rows=0), FFN) == B.MOE_OK
    assert call("moe_ffn_grad", ffn(rows=0), FFN_GRAD[:14] + [0, 0, 0, P]) == B.MOE_OK


def norm(T=4, H=128, fp32=0, gate=2, eps=1e-6, alpha=1.0):
    return B.MoeNormDesc(T, H, fp32, gate, eps, alpha)


NORM = [P] * 8        # x, o, w_post, gate, w_pre, r, n, err
NORM_GRAD = [P] * 14  # r, o, w_post, gate, w_pre, grad_r, grad_n, grad_x, grad_o, 3 vectors, workspace, err


@pytest.mark.parametrize("d", [norm(T=-1), norm(H=0), norm(H=12), norm(H=32776), norm(fp32=2), norm(gate=3),
                               norm(eps=-1e-6), norm(eps=float("nan")), norm(eps=float("inf")),
                               norm(alpha=float("inf")), norm(alpha=float("nan"))])
def test_norm_refuses_sizes(d):
    assert call("moe_norm", d, NORM) == B.MOE_EINVAL
    assert call("moe_norm_grad", d, NORM_GRAD) == B.MOE_EINVAL
    with pytest.raises(B.MoeError):
        B.moe_norm_workspace(d)


# o, w_post and the stream's gradient may be missing: what depends on them is then refused by itself
@pytest.mark.parametrize("at,value", [(i, P + 2) for i in range(8)] + [(i, 0) for i in (0, 1, 3, 4, 5, 6, 7)])
def test_norm_refuses_missing_or_unaligned_buffers(at, value):
    args = list(NORM)
    args[at] = value
    assert call("moe_norm", norm(), args) == B.MOE_EINVAL


@pytest.mark.parametrize("at,value", [(i, P + 2) for i in range(14)] + [(i, 0) for i in range(14) if i not in (2, 5)])
def test_norm_grad_refuses_missing_or_unaligned_buffers(at, value):
    args = list(NORM_GRAD)
    args[at] = value
    assert call("moe_norm_grad", norm(), args) == B.MOE_EINVAL


def test_norm_workspace():
    assert B.moe_norm_workspace(norm(T=0)) == 0
    assert B.moe_norm_workspace(norm(T=3)) == 3 * 2 * 128 * 4
    assert B.moe_norm_workspace(norm(T=100000)) == B.moe_norm_workspace(norm(T=200000))
