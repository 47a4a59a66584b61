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


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("H", [96, 320, 4096])
def test_non_finite_stays_in_its_row(bad, H):
    """With a checkpoint: the other rows keep their y, statistics, codes and
    gradients; the row itself has NaN (its mean: what its sum gives)."""
    say(f"layernorm with {bad} and a checkpoint H={H}")
    T, row, g = 40, 11, torch.Generator().manual_seed(H)
    x, dy = torch.randn(T, H, generator=g).to(BF).cuda(), torch.randn(T, H, generator=g).to(BF).cuda()
    y0, s0 = moe.moe_layernorm_fwd(x, checkpoint=True)
    d0 = moe.moe_layernorm_bwd(dy, s0)[0]
    x[row, H - 7] = bad
    y1, s1 = moe.moe_layernorm_fwd(x, checkpoint=True)
    d1 = moe.moe_layernorm_bwd(dy, s1)[0]
    d2 = moe.moe_layernorm_bwd(dy, s1 | {"xhat_codes": None, "xhat_scales": None}, x=x)[0]
    d3 = moe.moe_layernorm_bwd(dy, s0 | {"xhat_codes": None, "xhat_scales": None}, x=x.nan_to_num(0, 0, 0))[0]
    torch.cuda.synchronize()
    keep = torch.arange(T, device="cuda") != row
    for a, b in ((y1, y0), (d1, d0), (d2, d3), *((s1[k], s0[k]) for k in s0 if k != "x_type")):
        assert torch.equal(a[keep], b[keep])
    assert y1[row].isnan().all() and s1["rstd"][row].isnan() and d2[row].isnan().all()
    assert not s1["mean"][row].isfinite()


@pytest.mark.parametrize("wt", [BF, F32], ids=["w_bf16", "w_f32"])
def test_one_weight_alone(wt):
    """gamma without beta and beta without gamma: as with the other one's neutral values."""
    say(f"layernorm with one weight w={wt}")
    g = torch.Generator().manual_seed(3)
    x, dy = torch.randn(70, 160, generator=g).to(BF).cuda(), torch.randn(70, 160, generator=g).to(BF).cuda()
    w = (1 + 0.2 * torch.randn(160, generator=g)).to(wt).cuda()
    one, zero = torch.ones_like(w), torch.zeros_like(w)
    assert torch.equal(moe.moe_layernorm_fwd(x, w)[0], moe.moe_layernorm_fwd(x, w, zero)[0])
    assert torch.equal(moe.moe_layernorm_fwd(x, None, w)[0], moe.moe_layernorm_fwd(x, one, w)[0])
    _, s = moe.moe_layernorm_fwd(x)
    a, b = moe.moe_layernorm_bwd(dy, s, None, x=x), moe.moe_layernorm_bwd(dy, s, torch.ones(160, device="cuda"), x=x)
    torch.cuda.synchronize()
    assert a[1].dtype == F32 and all(torch.equal(p, q) for p, q in zip(a, b))


def test_squares_past_the_range():
    """Deviations whose squares leave fp32: rstd and xh are 0, y is beta, in those rows alone."""
    say("layernorm with squares past fp32")
    x = torch.randn(6, 256, generator=torch.Generator().manual_seed(4))
    clean, s0 = moe.moe_layernorm_fwd(x.cuda(), checkpoint=True)
    x[2] *= 2.0 ** 100
    beta = torch.full((256,), 0.5, device="cuda")
    y, s = moe.moe_layernorm_fwd(x.cuda(), checkpoint=True)
    z, _ = moe.moe_layernorm_fwd(x.cuda(), None, beta)
    torch.cuda.synchronize()
    keep = torch.arange(6) != 2
    assert torch.equal(y.cpu()[keep], clean.cpu()[keep])
    assert s["rstd"][2] == 0 and not y[2].any() and (z[2] == 0.5).all() and not s["xhat_scales"][2].any()
