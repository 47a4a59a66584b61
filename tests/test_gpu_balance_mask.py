"""GPU: a masked balance loss whose backward is called with what the forward saved, and nothing else."""
import pytest
import torch

import mxfp8_block_scaled_top_amd as moe
from oracle import block8 as B
from tests.helpers import need_gpu, say
from tests.test_gpu_balance import U, _case

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    need_gpu()


@pytest.mark.parametrize("dtype", [torch.bool, torch.uint8])
@pytest.mark.parametrize("T,E,k", [(1, 4, 1), (300, 8, 2), (1500, 61, 3)])
def test_backward_without_the_mask_uses_the_forwards(T, E, k, dtype):
    say(f"balance backward, saved mask T={T} E={E} {dtype}")
    x, topk, mask, d0 = _case(T, E, k, seed=T, masked=True, add=True)
    m = mask.to(dtype).cuda()
    _, saved = moe.moe_balance_fwd(x.cuda(), topk.cuda(), m, 0.1, 0.01)
    given = moe.moe_balance_bwd(x.cuda(), saved, m, dlogits=d0.cuda())
    alone = moe.moe_balance_bwd(x.cuda(), saved, dlogits=d0.cuda())
    torch.cuda.synchronize()
    assert torch.equal(alone, given)
    assert torch.equal(alone.cpu()[~mask], d0[~mask])           # a token that does not count adds nothing
    r = B.balance(x, topk, mask, 0.1, 0.01)
    # terms of a row at most as large as these, some 60 roundings (the bound of test_gpu_balance, coarser)
    n = max(1, r["tokens"])
    size = 0.1 * E / n * r["p"] * (r["f"] + 1) + 0.02 / n * r["lse"].abs()[:, None] * r["p"]
    assert ((alone.cpu().double() - (r["dlogits"] + d0.double())).abs() <= 128 * U * size + U * 4 * d0.abs() + 1e-37).all()


def test_without_a_mask_every_token_counts():
    say("balance backward, no mask")
    x, topk, mask, _ = _case(40, 8, 2, seed=1, masked=True)
    _, saved = moe.moe_balance_fwd(x.cuda(), topk.cuda(), None, 0.1, 0.01)
    d = moe.moe_balance_bwd(x.cuda(), saved)
    torch.cuda.synchronize()
    assert (d != 0).any(1).all()
