"""GPU: RMS norm with more rows than the workgroups of a launch hold at once, at every kernel shape, so that each
workgroup goes on to further rows (the next row's loads, gamma's sums over rows, the buffers used in turn).
Bounds as in test_gpu_rmsnorm."""
import pytest
import torch

from tests.helpers import need_gpu, say
from tests.test_gpu_rmsnorm import BF, F32, _bwd_case, _fwd_case

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    need_gpu()


# rows at once: 4096 up to 1024 columns (8192 and more up to 256), 1024 to 2048 up to 2048, 512 to 1024 up to 4096,
# 256 to 512 up to 8192, 256 beyond; the last sizes of a shape and ones whose last lanes have nothing
SIZES = [(17000, 64), (9001, 248), (4500, 512), (4300, 456), (4500, 1000), (2500, 2048), (2600, 1416), (1100, 4096),
         (1200, 2312), (600, 8192), (1100, 5000), (600, 8200), (600, 16384), (300, 16392), (300, 32768)]


@pytest.mark.parametrize("T,H", SIZES)
@pytest.mark.parametrize("xt,st,wt", [(BF, BF, F32), (F32, F32, BF), (BF, F32, None)], ids=["bf16", "f32", "mixed"])
def test_forward(T, H, xt, st, wt):
    say(f"rmsnorm fwd, further rows T={T} H={H} x={xt} stream={st}")
    _fwd_case(T, H, xt, st, wt, st != xt or xt == BF, True, seed=T)


@pytest.mark.parametrize("T,H", SIZES)
@pytest.mark.parametrize("st,wt,res,branch", [(BF, BF, False, False), (F32, F32, True, True)], ids=["bf16", "f32_res_branch"])
def test_backward(T, H, st, wt, res, branch):
    say(f"rmsnorm bwd, further rows T={T} H={H} stream={st}")
    _bwd_case(T, H, st, wt, res, branch, seed=T)


@pytest.mark.parametrize("st", [BF, F32])
def test_backward_past_the_most_partial_rows(st):
    """Above 8192 columns gamma's gradient has its own kernel, 4 rows a workgroup and at most 60 partial rows for
    8200 columns: 300 rows give each workgroup a second set."""
    say(f"rmsnorm bwd, 300 x 8200 {st}")
    _bwd_case(300, 8200, st, F32, False, False, seed=3)
    _bwd_case(1, 8200, st, F32, False, False, seed=4)
