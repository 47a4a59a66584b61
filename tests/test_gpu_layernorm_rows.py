"""GPU: layer norm batches in which every workgroup walks over several groups of
rows, for each width that has a kernel shape of its own, against float64 with the
bounds of test_gpu_layernorm.py: dgamma and dbeta carried over the rows, the sums'
LDS used again from row to row, the next row loaded ahead (or not, above 16384)
and, above 8192, the kernel of the weights' gradients over several rows and
partial rows.

The chain of additions that those bounds count for a weight's gradient (T / 512 + 68)
holds here too: a thread adds at most T / 256 < 4 rows of its own (the column kernel
T / 64 < 10), the workgroup 8 partial sums, the second kernel 8 and 18 more."""
import pytest
import torch

from tests import test_gpu_layernorm as L
from tests.helpers import need_gpu, say

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(autouse=True)
def _gpu():
    need_gpu()


# rows at once: forward 4096, 4096, 4096, 2048, 2048, 1024, 512, 256, 256, 256, 256
FWD = [(9001, 504), (9001, 512), (9003, 640), (5003, 1416), (5003, 2048), (2309, 4096), (1201, 8192), (601, 8200),
       (601, 16384), (300, 16392), (300, 32768)]
# backward 4096, 4096, 2048, 1024, 1024, 512, 256, 256, 256, 256, 256
BWD = [(9001, 504), (9001, 512), (5003, 640), (2309, 1416), (3085, 2048), (1201, 4096), (701, 8192), (601, 8200),
       (601, 16384), (300, 16392), (300, 32768)]


@pytest.mark.parametrize("T,H", FWD)
@pytest.mark.parametrize("xt,wt", [(BF, F32), (F32, BF)], ids=["bf16", "f32"])
def test_forward(T, H, xt, wt):
    say(f"layernorm fwd over several rows T={T} H={H} x={xt}")
    L._fwd_case(T, H, xt, wt, ckpt=H % 32 == 0, seed=H + 1)


@pytest.mark.parametrize("T,H", BWD)
@pytest.mark.parametrize("xt,wt,res", [(BF, F32, False), (F32, BF, True)], ids=["bf16", "f32_res"])
def test_backward(T, H, xt, wt, res):
    say(f"layernorm bwd over several rows T={T} H={H} x={xt} res={res}")
    L._bwd_case(T, H, xt, wt, False, res, seed=H + 1)


@pytest.mark.parametrize("T,H", [s for s in BWD if s[1] % 32 == 0])
@pytest.mark.parametrize("xt,wt,res", [(BF, BF, True), (F32, F32, False)], ids=["bf16_res", "f32"])
def test_backward_from_checkpoint(T, H, xt, wt, res):
    say(f"layernorm bwd from 8 bits over several rows T={T} H={H} x={xt} res={res}")
    L._bwd_case(T, H, xt, wt, True, res, seed=H + 1)
