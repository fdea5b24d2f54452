"""moe_lora_linear with any num_sms that the header allows: more SMs than there are count as all of them."""
import ctypes
import subprocess
import sys

import pytest
import torch

from combine_moe_layout_gb300 import _binding as B

CALL = """
import ctypes, sys
from combine_moe_layout_gb300 import _binding as B
p = ctypes.c_void_p(1 << 20)
d = B.MoeLoraDesc(int(sys.argv[1]), 64, 64, 16, 0, int(sys.argv[2]))
st = B.load().moe_lora_linear(ctypes.byref(d), p, p, None, None, None, None, None, p, p, None)
sys.exit(0 if st == B.MOE_ECUDA else 3)
"""


@pytest.mark.skipif(torch.cuda.is_available(), reason="the addresses are not to be read")
@pytest.mark.parametrize("T", [1, 40])
@pytest.mark.parametrize("num_sms", [0, 1, 1 << 30, 2 ** 31 - 1])
def test_the_call_returns(T, num_sms):
    """In a process of its own, since a division by zero would end it. Without a device the launch is what fails."""
    r = subprocess.run([sys.executable, "-c", CALL, str(T), str(num_sms)], timeout=300)
    assert r.returncode == 0


@pytest.mark.gpu
@pytest.mark.parametrize("num_sms", [152, 1000, 1 << 30, 2 ** 31 - 1])
@pytest.mark.parametrize("T,A", [(1, 0), (1, 3), (40, 2), (130, 3), (700, 2)])
def test_more_sms_than_there_are(T, A, num_sms):
    """The same bits as with all SMs: the same tiles, splits and order of sums."""
    from test_gpu_lora import bf16, ids_of, run
    from gpu_common import require_gpu
    require_gpu()
    assert num_sms >= torch.cuda.get_device_properties(0).multi_processor_count
    K, N, r = 264, 520, 24
    x, w = bf16((T, K), 1), bf16((N, K), 2, K ** -0.5)
    la, lb = (bf16((A, r, K), 3, K ** -0.5), bf16((A, N, r), 4, r ** -0.5)) if A else (None, None)
    ids = ids_of(T, A, "tokens") if A else None
    want, st = run(x, w, la, lb, None, ids)
    got, st2 = run(x, w, la, lb, None, ids, num_sms=num_sms)
    assert st == st2 == B.MOE_OK and torch.equal(got, want)
