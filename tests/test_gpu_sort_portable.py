"""The ranking in clusters of at most eight CTAs, which every device grants: what moe_sort falls back to where sixteen
find no room. The sort is built once more with that limit, and gives the same bits."""
from __future__ import annotations

import ctypes
import os
import subprocess

import pytest
import torch

from combine_moe_layout_gb300 import _binding as B
from combine_moe_layout_gb300 import _build
from gpu_common import require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def portable(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("portable") / "libsort.so")
    src = [os.path.join(_build.CSRC, f) for f in ("moe_sort.cu", "moe_combine.cu", "moe_layout.cu")]
    subprocess.run([_build.nvcc(), *_build.NVCC_FLAGS, "-DMOE_RANK_CLUSTER=8", "-shared", "-t", "3", "-o", so, *src],
                   check=True)
    fn = ctypes.CDLL(so).moe_sort
    fn.restype = ctypes.c_int32
    return fn


@pytest.mark.parametrize("T,E,k,masked", [(600, 8, 8, 0.0), (8192, 256, 8, 0.1), (40001, 1000, 3, 0.0), (9000, 8192, 1, 0.3)])
def test_eight_ctas_give_what_sixteen_give(portable, T, E, k, masked):
    require_gpu()
    g = torch.Generator(device="cuda:0").manual_seed(T)
    idx = torch.randint(0, E, (T, k), generator=g, device="cuda:0", dtype=torch.int32)
    idx.masked_fill_(torch.rand((T, k), generator=g, device="cuda:0") < masked, -1)
    x = torch.randn((T, 8), generator=g, device="cuda:0").to(torch.bfloat16)
    d = B.MoeDesc(1, T, 8, E, k, T, B.MOE_BF16, 0)
    err = torch.zeros(1, dtype=torch.int32, device="cuda:0")
    got = []
    for fn in (B.load().moe_sort, portable):
        out = [torch.zeros(E + 1, dtype=torch.int32, device="cuda:0"),
               torch.zeros((T * k, 8), dtype=torch.bfloat16, device="cuda:0"),
               torch.zeros((T, k), dtype=torch.int32, device="cuda:0")]
        off, px, tok = (ctypes.c_void_p(t.data_ptr()) for t in out)
        st = fn(ctypes.byref(d), ctypes.c_void_p(idx.data_ptr()), ctypes.c_void_p(x.data_ptr()), None, off, px, None, tok,
                ctypes.c_void_p(err.data_ptr()), ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
        assert st == B.MOE_OK and B.moe_get_error(err) == B.MOE_OK
        got.append(out)
    assert all(torch.equal(a, b) for a, b in zip(*got))
