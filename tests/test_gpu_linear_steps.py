"""bf16 grouped_linear at K extents that end inside a pair of the GEMM's K steps
(an odd number of blocks of 32) and at every count of steps up to a few rounds of
its pipeline, against the product in 64 bits.  Forward (both operands contiguous
along K), dX (K is N there) and dW (K is the rows)."""
import pytest
import torch

import mxfp8_block_scaled_top_amd as moe
from tests.helpers import need_gpu, say

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    need_gpu()


def _near(got, a, b, what):
    """got = round(a b): half a bf16 step of the value, and fp32 products summed
    in K + 1 roundings of at most 2^-24 of the sum of magnitudes each."""
    a, b = a.double(), b.double()
    want, mag = a @ b, a.abs() @ b.abs()
    tol = (2.0 ** -8 * want.abs() + (a.shape[1] + 1) * 2.0 ** -24 * mag) * (1 + 2.0 ** -7)
    bad = (got.double() - want).abs() > tol
    assert not bad.any(), (what, int(bad.sum()), bad.nonzero()[:3].tolist())


@pytest.mark.parametrize("blocks", [1, 2, 3, 4, 5, 6, 7, 9, 12, 13])
@pytest.mark.parametrize("sizes,N", [((1,), 32), ((70, 0, 301), 96), ((257,), 288)])
def test_linear_at_every_count_of_steps(blocks, sizes, N):
    K, rows = 32 * blocks, sum(sizes)
    say(f"linear steps: sizes={sizes} N={N} K={K}")
    g = torch.Generator().manual_seed(rows + N + K)
    # exact sizes: the operands' last rows end where their storage ends
    x = torch.randn(rows, K, generator=g).bfloat16()
    dy = torch.randn(rows, N, generator=g).bfloat16()
    w = [torch.randn(N, K, generator=g).bfloat16() for _ in sizes]
    sp = torch.tensor(sizes, dtype=torch.int32).cuda()
    wd = [t.cuda() for t in w]
    y = moe.grouped_linear_fwd(x.cuda(), sp, wd).cpu()
    dx, dw = moe.grouped_linear_bwd(dy.cuda(), x.cuda(), sp, wd)
    r = 0
    for e, m in enumerate(sizes):
        s = slice(r, r + m)
        _near(y[s], x[s], w[e].T, ("y", e))
        _near(dx[s].cpu(), dy[s], w[e], ("dx", e))
        _near(dw[e].cpu(), dy[s].T, x[s], ("dw", e))
        r += m


@pytest.mark.parametrize("N", [32, 64, 96, 160, 416])
def test_linear_dx_at_every_count_of_steps(N):
    """dX sums over N: the same extents for its operands (dY along N, W as it lies)."""
    sizes, K = (33, 200), 64
    say(f"linear dx steps: N={N}")
    g = torch.Generator().manual_seed(N)
    x = torch.randn(sum(sizes), K, generator=g).bfloat16()
    dy = torch.randn(sum(sizes), N, generator=g).bfloat16()
    w = [torch.randn(N, K, generator=g).bfloat16() for _ in sizes]
    dx, _ = moe.grouped_linear_bwd(dy.cuda(), x.cuda(), torch.tensor(sizes, dtype=torch.int32).cuda(),
                                   [t.cuda() for t in w], want_dw=False)
    _near(dx[:33].cpu(), dy[:33], w[0], "dx 0")
    _near(dx[33:].cpu(), dy[33:], w[1], "dx 1")
