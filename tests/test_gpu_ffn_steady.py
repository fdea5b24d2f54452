"""The feed-forward block where its kernels' loops come round: refills of the few-row kernel, clusters of every size and
checkpoints in 8 bits in them, more than two tiles to a CTA in every form, many experts. Bars as in test_gpu_ffn."""
import pytest
import torch

from combine_moe_layout_gb300 import _binding as B
from test_gpu_ffn import Case

pytestmark = pytest.mark.gpu
SAVED = [B.MOE_SAVE_BF16, B.MOE_SAVE_FP8]
MOST = 2048  # MOE_FFN_MAX_EXPERTS


def both_ways(c):
    c.forward()
    c.check_forward()
    c.keep_made()
    c.backward()
    c.check_backward()


@pytest.mark.parametrize("rows", [1, 8, 9, 16])
@pytest.mark.parametrize("H,I", [(1800, 1032), (4096, 520), (520, 4104)])
@pytest.mark.parametrize("save", [B.MOE_SAVE_NONE, B.MOE_SAVE_BF16])
def test_few_rows_of_wide_blocks(rows, H, I, save):
    """A warp takes the K chunks of 32 in turns of 8 x 7, or 8 x 4 with more than 8 rows: a second turn begins at a width
    of 1792, or 1024."""
    c = Case([rows], H, I, save=save, dense=True)
    c.forward()
    c.check_forward()


@pytest.mark.parametrize("counts", [[0, 3, 0, 2, 1], [1] * 16, [0] * 260 + [4, 0, 5] + [0] * 36 + [1]])
def test_few_rows_of_experts(counts):
    """The last: more experts than the kernel has threads."""
    c = Case(counts, 2056, 264, B.MOE_ACT_GELU_TANH, behind=2 if sum(counts) < 15 else 0, ranks=2)
    c.forward()
    c.check_forward()


@pytest.mark.parametrize("save", SAVED)
@pytest.mark.parametrize("num_sms", [16, 24, 32, 40, 48, 56, 64, 96, 128, 0])
def test_clusters_of_every_size(num_sms, save):
    """16 tiles in linear 1 and 8 in the other three forms, so that num_sms / 16 and num_sms / 8 CTAs share one, up to 8."""
    both_ways(Case([100], 2048, 2048, save=save, behind=3, num_sms=num_sms))


@pytest.mark.parametrize("save", SAVED)
@pytest.mark.parametrize("act", [B.MOE_ACT_SILU, B.MOE_ACT_GELU_TANH])
@pytest.mark.parametrize("counts,H,I", [([70, 0, 33, 5, 128, 1], 1032, 512), ([129, 17], 1544, 640), ([40], 4096, 128)])
def test_ragged_batches_in_clusters(counts, H, I, act, save):
    both_ways(Case(counts, H, I, act, save, behind=2, seed=3))


@pytest.mark.parametrize("save", SAVED)
@pytest.mark.parametrize("counts,H,I", [([300, 0, 201, 40], 264, 384), ([64] * 9, 512, 256)])
def test_several_tiles_to_a_cta_in_every_form(counts, H, I, save):
    """Two CTAs: each accumulator is taken again, and those of 8 bits are read twice before they are given back."""
    both_ways(Case(counts, H, I, save=save, behind=1, num_sms=2, seed=4))


@pytest.mark.parametrize("tail", [1, 15, 16, 17, 33, 63])
def test_tails_beside_rows_that_are_not_finite(tail):
    """The weights' gradient of an expert whose last K block holds `tail` rows of its own and the next one's behind."""
    c = Case([64 + tail, 70], 264, 200, save=B.MOE_SAVE_BF16, behind=3, seed=5)
    c.keep_made()
    for t in (c.x, c.grad_y, c.gate, c.up):
        t[64 + tail:] = float("nan")
    c.backward()
    c.check_backward(experts=[0])


def test_the_most_experts():
    counts = [0] * MOST
    for i in range(0, MOST, 93):
        counts[i] = 1 + i % 140
    counts[-1] = 65
    c = Case(counts, 136, 72, save=B.MOE_SAVE_BF16, behind=2, seed=6)
    used = [e for e, n in enumerate(counts) if n]
    c.forward()
    c.check_forward()
    c.keep_made()
    c.backward()
    c.check_backward(experts=used)
    empty = torch.tensor([n == 0 for n in counts])
    assert not any(bool(t[empty.to(t.device)].any()) for t in c.gw)
