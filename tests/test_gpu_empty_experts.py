"""GPU: weight gradients of experts without rows are zeros, in buffers that held
something else, and nothing past them is written: at widths that end inside a tile."""
import ctypes

import pytest
import torch

import mxfp8_block_scaled_top_amd as moe
from tests.helpers import need_gpu, say

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


@pytest.fixture(autouse=True)
def _gpu():
    need_gpu()


@pytest.mark.parametrize("precision", [moe.MOE_BF16, moe.MOE_MXFP8], ids=["bf16", "mxfp8"])
@pytest.mark.parametrize("N,K", [(32, 32), (96, 288), (288, 96), (544, 2080), (2048, 1056), (2304, 256)])
@pytest.mark.parametrize("sizes", [(0, 5, 0), (0, 0, 70, 0), (0, 0)])
def test_grouped_linear(precision, N, K, sizes):
    say(f"empty experts N={N} K={K} sizes={sizes} precision={precision}")
    rows, E, pad = sum(sizes), len(sizes), 512
    g = torch.Generator().manual_seed(N + K + rows)
    x, dy = torch.randn(rows, K, generator=g).to(BF).cuda(), torch.randn(rows, N, generator=g).to(BF).cuda()
    w = [torch.randn(N, K, generator=g).to(BF).cuda() for _ in sizes]
    split = torch.tensor(sizes, dtype=torch.int32).cuda()
    dw = [torch.full((N * K + pad,), 7.0, dtype=BF, device="cuda") for _ in sizes]
    n = moe.moe_workspace_bytes(moe.MOE_OP_LINEAR_BWD, rows, K, N, E, 1, precision)
    ws = torch.empty(max(n, 256), dtype=torch.uint8, device="cuda")
    table = lambda ts: (ctypes.c_void_p * E)(*[t.data_ptr() for t in ts])                # noqa: E731
    p = lambda t: t.data_ptr() or None                                                  # noqa: E731
    assert moe.lib().grouped_linear_bwd(precision, E, N, K, rows, p(dy), p(x), p(split), table(w), None, table(dw),
                                        p(ws), ws.numel(), torch.cuda.current_stream().cuda_stream) == 0
    torch.cuda.synchronize()
    for e, m in enumerate(sizes):
        assert (dw[e][N * K:] == 7).all(), e
        if m == 0:
            assert not dw[e][:N * K].any(), e
        else:
            want = dy.double().T @ x.double()
            d = dw[e][:N * K].view(N, K).double() - want
            # half a bf16 step; E4M3 codes are off by 0.026 in the mean square (at most
            # 2^-4), two operands by 0.037 of the product, held to twice that
            assert float(d.norm()) <= (2.0 ** -8 if precision == moe.MOE_BF16 else 0.08) * float(want.norm()), e
