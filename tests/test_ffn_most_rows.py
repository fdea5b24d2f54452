"""How many rows and columns the feed-forward block takes, on the host alone: a tile that begins before the last of them
ends up to 255 behind it, and they are counted in 32 bits. (Refused before any launch, so that no pointer is followed;
without a device a call that is not refused ends with MOE_ECUDA.)"""
import ctypes

import pytest

from combine_moe_layout_gb300 import _binding as B

P = 1 << 20  # an aligned address that is never read
MOST = 2 ** 31 - 1


def refused(name, count, rows, hidden=8, inter=8):
    d = B.MoeFfnDesc(rows, hidden, inter, 1, 1, 0, 1, 0)
    a = [ctypes.c_void_p(P)] * count + [ctypes.c_void_p(None)]
    return getattr(B.load(), name)(ctypes.byref(d), *a) == B.MOE_EINVAL


@pytest.mark.parametrize("name,count", [("moe_ffn", 12), ("moe_ffn_grad", 18)])
def test_a_last_tile_that_passes_32_bits_is_refused(name, count):
    assert refused(name, count, MOST) and refused(name, count, MOST - 127)
    assert refused(name, count, 100, hidden=MOST - 7) and refused(name, count, 100, inter=MOST - 7)
