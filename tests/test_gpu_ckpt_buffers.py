"""GPU: the checkpointed grouped MLP given saved tensors of other sizes (refused
before any launch, larger ones accepted with the same results) and a larger
batch's workspace."""
import pytest
import torch

import mxfp8_block_scaled_top_amd as moe
from tests.helpers import need_gpu, say

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
ALL, IDS = [moe.MOE_BF16, moe.MOE_MXFP8, moe.MOE_FP8], ["bf16", "mxfp8", "fp8"]


@pytest.fixture(autouse=True)
def _gpu():
    need_gpu()


def _inputs(sizes, H, I, seed):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s, std=1.0: (torch.randn(*s, generator=g) * std).to(BF).cuda()     # noqa: E731
    rows, E = sum(sizes), len(sizes)
    args = (torch.tensor(sizes, dtype=torch.int32).cuda(), [r(2 * I, H, std=0.05) for _ in range(E)],
            [r(H, I, std=0.05) for _ in range(E)], torch.rand(rows, generator=g).cuda())
    return r(rows, H), r(rows, H), args


@pytest.mark.parametrize("precision", ALL, ids=IDS)
def test_saved_of_other_sizes(precision):
    sizes, H, I = [40, 0, 25], 256, 384
    rows, E = sum(sizes), len(sizes)
    say(f"mlp ckpt saved sizes precision={precision}")
    xp, dyp, args = _inputs(sizes, H, I, 1)
    yp, saved = moe.grouped_mlp_fwd_ckpt(xp, *args, precision)
    want = moe.grouped_mlp_bwd_ckpt(dyp, xp, *args, saved, precision)
    bad = [saved | {k: saved[k].cpu()} for k in saved]
    if precision == moe.MOE_BF16:
        bad += [saved | {"a2": saved["a2"][:-1]}, saved | {"a2": saved["a2"].float()}]
    else:       # A1's tensors depend on neither H nor E: they have the right shapes
        bad += [moe.alloc_saved(rows, 128, I, E, precision, "cuda", checkpoint=True),
                moe.alloc_saved(rows, H, I, 1, precision, "cuda", checkpoint=True)]
    for s in bad:
        with pytest.raises(moe.MoEError):
            moe.grouped_mlp_fwd_ckpt(xp, *args, precision, s)
        with pytest.raises(moe.MoEError):
            moe.grouped_mlp_bwd_ckpt(dyp, xp, *args, s, precision)
    # longer buffers beside A1's
    big = moe.alloc_saved(2 * rows, 2 * H, I, 2 * E, precision, "cuda", checkpoint=True)
    big |= {k: torch.empty_like(saved[k]) for k in ("a1_codes", "a1_scales")}
    y2, _ = moe.grouped_mlp_fwd_ckpt(xp, *args, precision, big)
    got = moe.grouped_mlp_bwd_ckpt(dyp, xp, *args, big, precision)
    torch.cuda.synchronize()
    assert torch.equal(yp, y2) and torch.equal(got[0], want[0]) and torch.equal(got[3], want[3])
    for e in range(E):
        assert torch.equal(got[1][e], want[1][e]) and torch.equal(got[2][e], want[2][e])


@pytest.mark.parametrize("precision", ALL, ids=IDS)
def test_workspace_of_a_larger_batch(precision):
    """One workspace for the largest batch, on either side of the few-row rule."""
    H, I, E, most = 128, 16640, 2, 130          # the rule takes up to 128 rows
    say(f"mlp ckpt workspace of {most} rows precision={precision}")
    bytes_ = [moe.moe_workspace_bytes(op, most, H, I, E, 1, precision)
              for op in (moe.MOE_OP_MLP_FWD, moe.MOE_OP_MLP_BWD)]
    ws = [torch.empty(max(n, 256), dtype=torch.uint8, device="cuda") for n in bytes_]
    for sizes in ([66, 64], [64, 64], [100, 0], [1, 0], [0, 0]):
        xp, dyp, args = _inputs(sizes, H, I, 2)
        yp, saved = moe.grouped_mlp_fwd_ckpt(xp, *args, precision, workspace=ws[0])
        got = moe.grouped_mlp_bwd_ckpt(dyp, xp, *args, saved, precision, ws[1])
        y2, _ = moe.grouped_mlp_fwd_ckpt(xp, *args, precision)
        want = moe.grouped_mlp_bwd_ckpt(dyp, xp, *args, saved, precision)
        torch.cuda.synchronize()
        assert torch.equal(yp, y2) and torch.equal(got[0], want[0]) and torch.equal(got[3], want[3])
        assert all(torch.equal(a, b) for k in (1, 2) for a, b in zip(got[k], want[k]))


@pytest.mark.parametrize("precision", ALL[1:], ids=IDS[1:])
def test_without_the_weights_copies(precision):
    """saved without the weights' columnwise copies: the backward makes them itself."""
    sizes, H, I = [300, 0, 45], 256, 384
    say(f"mlp ckpt without weight copies precision={precision}")
    xp, dyp, args = _inputs(sizes, H, I, 3)
    yp, saved = moe.grouped_mlp_fwd_ckpt(xp, *args, precision)
    bare = moe.alloc_saved(sum(sizes), H, I, len(sizes), precision, "cuda", weight_cols=False, checkpoint=True)
    y2, bare = moe.grouped_mlp_fwd_ckpt(xp, *args, precision, bare)
    want = moe.grouped_mlp_bwd_ckpt(dyp, xp, *args, saved, precision)
    got = moe.grouped_mlp_bwd_ckpt(dyp, xp, *args, bare, precision)
    torch.cuda.synchronize()
    assert torch.equal(yp, y2) and torch.equal(got[0], want[0]) and torch.equal(got[3], want[3])
    assert all(torch.equal(a, b) for k in (1, 2) for a, b in zip(got[k], want[k]))
