"""The GEMMs that make and read 8-bit checkpoints on wide tiles and on narrow
tiles that follow one another: the checks of ragged buffers (plain training
forward's G | U to its codes bit by bit, the backward against 64 bits) at sizes
that take them."""
import pytest
import torch

import mixture_experts_layer_fp32_amd as moe
from test_gpu_ckpt import test_backward_from_codes as backward_from_codes
from test_gpu_ckpt import test_training_forward_codes as training_forward_codes

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu_and_library():
    assert torch.cuda.is_available(), "no GPU visible"
    moe.load_library()
    yield
    torch.cuda.synchronize()


# Wide tiles (256 rows x 128 columns, where they need one round of workgroups
# and narrow ones two): several column tiles, the last one half, long K, row
# blocks of every size.
WIDE = [([300, 1, 0, 513], 1088, 320, 20000), ([255, 257, 512], 448, 192, 28000),
        ([1, 600, 33, 0, 2], 192, 1024, 7000), ([1000], 128, 192, 30000),
        ([900, 1100, 1200, 700, 1090], 64, 1024, None)]
# Narrow tiles, more than one a workgroup.
NARROW = [([int(i * 37 % 101) for i in range(70)], 128, 448, 7000),
          ([int(i * 53 % 131) for i in range(70)], 320, 448, None)]


@pytest.mark.parametrize("wide,cases", [(True, WIDE), (False, NARROW)])
def test_cases_take_the_tiles_they_are_for(wide, cases):
    for counts, D, I, cap in cases:
        n, rows = len(counts), sum(counts) if cap is None else cap
        d = moe.make_desc(T=rows, D=D, E=n, top_k=1, I=I)
        assert moe.moe_ffn_tile_shape(d, n, I, rows, True, 0) == ((256, 256) if wide else (320, 128))


@pytest.mark.parametrize("counts,D,I,cap", WIDE + NARROW)
def test_training_forward_codes(counts, D, I, cap):
    training_forward_codes(counts, D, I, cap)


@pytest.mark.parametrize("counts,D,I,cap", WIDE + NARROW)
def test_backward_from_codes(counts, D, I, cap):
    backward_from_codes(counts, D, I, cap)
