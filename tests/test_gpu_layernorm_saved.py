"""GPU: what the layer norm's backward takes from the forward's saved tensors."""
import pytest
import torch

import mxfp8_block_scaled_top_amd as moe
from tests.helpers import need_gpu, say

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(autouse=True)
def _gpu():
    need_gpu()


@pytest.mark.parametrize("xt", [BF, F32], ids=["bf16", "f32"])
def test_gradient_has_the_type_of_the_forwards_x(xt):
    """From a checkpoint alone: an fp32 residual stream gets an fp32 gradient."""
    say(f"layernorm dx type from the checkpoint x={xt}")
    g = torch.Generator().manual_seed(1)
    x, dy = torch.randn(20, 96, generator=g).to(xt).cuda(), torch.randn(20, 96, generator=g).to(BF).cuda()
    _, saved = moe.moe_layernorm_fwd(x, checkpoint=True)
    want = moe.moe_layernorm_bwd(dy, saved, x=x)
    for kept in (saved, {k: t.clone() for k, t in saved.items()}):
        got = moe.moe_layernorm_bwd(dy, kept)
        torch.cuda.synchronize()
        assert got[0].dtype == xt and all(torch.equal(a, b) for a, b in zip(got, want))
    # an asked-for type and dres's come first; a dict without the entry gives bf16
    other = F32 if xt == BF else BF
    assert moe.moe_layernorm_bwd(dy, saved, dx_dtype=other)[0].dtype == other
    assert moe.moe_layernorm_bwd(dy, saved, dres=dy.to(other))[0].dtype == other
    del saved["x_type"]
    assert moe.moe_layernorm_bwd(dy, saved)[0].dtype == BF
