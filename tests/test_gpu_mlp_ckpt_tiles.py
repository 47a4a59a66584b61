"""GPU: the checkpointed grouped MLP at widths whose tile counts are multiples of
8, where the tiles go to the XCDs by other maps than elsewhere: column tiles of
every expert in turn (gate_up I / 128; the dgrads and dW_down I / 256, H / 256) and
dW_gate_up's row tiles (2I / 256).  The backward numbers two products' workgroups in
one grid; results are those of the separate launches, bit for bit."""
import pytest

import mxfp8_block_scaled_top_amd as moe
from tests import test_gpu_mlp_ckpt as M
from tests.helpers import need_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    need_gpu()


@pytest.mark.parametrize("precision", M.ALL, ids=M.IDS)
@pytest.mark.parametrize("sizes,H,I", [([700, 0, 1, 900, 300], 256, 1024), ([300, 257, 0, 600], 2048, 2048),
                                       ([513, 0, 300], 2048, 1024), ([1, 1100, 0, 30], 384, 2048)])
def test_against_the_separate_launches(precision, sizes, H, I):
    assert not M._few(moe.MOE_BF16, sizes, I)
    M.test_against_the_bf16_form(precision, sizes, H, I)
