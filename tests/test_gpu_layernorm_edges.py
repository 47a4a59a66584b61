"""GPU: layer norm rows at the ends of the number range and with values that are
not finite, against float64."""
import pytest
import torch

import mxfp8_block_scaled_top_amd as moe
from oracle import sublayer as S
from tests.helpers import need_gpu, say

pytestmark = pytest.mark.gpu

U, BF, F32 = 2.0 ** -24, torch.bfloat16, torch.float32
C = 64          # the longest chain of a row's sum: 32 values, 6 steps in a wave, 16 waves


@pytest.fixture(autouse=True)
def _gpu():
    need_gpu()


@pytest.mark.parametrize("H", [8, 64, 136, 264, 520, 1416, 2056, 4104, 8200, 16392])
@pytest.mark.parametrize("xt", [BF, F32], ids=["bf16", "f32"])
def test_constant_rows_of_large_values(H, xt):
    """x = mean = 2^120: xh is 0 and mean rstd is not a finite number.  The lanes
    past a row's end hold no x; whatever they hold adds nothing to the sums."""
    say(f"layernorm bwd of constant rows of 2^120 H={H} x={xt}")
    T, g = 5, torch.Generator().manual_seed(H)
    x = torch.full((T, H), 2.0 ** 120)
    dy = torch.randn(T, H, generator=g).to(BF)
    mean, rstd = torch.full((T,), 2.0 ** 120), torch.full((T,), 316.25)
    dx, dgamma, dbeta = moe.moe_layernorm_bwd(dy.cuda(), {"mean": mean.cuda(), "rstd": rstd.cuda()}, x=x.to(xt).cuda())
    torch.cuda.synchronize()
    r = S.layernorm_bwd(dy, torch.zeros(T, H), rstd)
    # mean(g): a chain of C additions and the division; the difference and the product round
    size = dy.double().abs()
    e = 316.25 * ((C + 3) * U * size.mean(1, keepdim=True) + 4 * U * (size + r["c1"].abs())) * 1.01
    half = 2.0 ** -8 if xt == BF else U
    assert ((dx.double().cpu() - r["dx"]).abs() <= e + half * (r["dx"].abs() + e)).all()
    assert not dgamma.any()
    assert ((dbeta.double().cpu() - r["dbeta"]).abs() <= (T + 64) * U * size.sum(0)).all()
