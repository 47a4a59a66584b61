"""GPU: block products whose two scales multiply to what fp32 does not hold although the values are in range.

Inputs are codes and scales as they are; a block's sum times the scales is compared with float64 under the bounds
of test_gpu_block_linear, which count the scales' product as one rounding: that holds where it has all of fp32's
bits, whatever its size.  Results below bf16's smallest normal number round to steps of 2^-133."""
import numpy as np
import pytest
import torch

import mxfp8_block_scaled_top_amd as moe
from oracle import block8 as B
from tests.helpers import need_gpu, say
from tests.test_gpu_block_linear import BF, H8, _product_bound

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    need_gpu()


def _within(got, ref, bound, what):
    d = (got.double().cpu() - ref).abs()
    lim = bound + H8 * (ref.abs() + bound) + 2.0 ** -134
    assert (d <= lim).all(), (what, float((d / lim).max()), float(ref.abs().max()))


def _case(rows, E, N, K, sx, sw, low, seed):
    """Codes of the top binade (256 .. 448; low: 1 .. 7 times 2^-9), scales near sx and sw with full mantissas."""
    g = np.random.default_rng(seed)
    span = (1, 8) if low else (0x78, 0x7F)
    xc, wc = (g.integers(*span, s).astype(np.uint8) for s in ((rows, K), (E, N, K)))
    nb, kb = (N + 127) // 128, (K + 127) // 128
    xs = (sx * (1 + g.random((kb, rows)))).astype(np.float32)
    ws = (sw * (1 + g.random((E, nb, kb)))).astype(np.float32)
    d = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()     # noqa: E731
    w8 = {"codes": d(wc), "scales": d(ws), "codes_t": d(wc.transpose(0, 2, 1))}
    return {"codes": d(xc), "scales": d(xs)}, w8, B.rows_value(xc, xs), [B.weight_value(c, s) for c, s in zip(wc, ws)]


# a full block of top codes sums to some 2^24, one of the lowest to 2^-7
PAIRS = [(2.0 ** -75, 2.0 ** -72, False), (2.0 ** -90, 2.0 ** -62, False), (2.0 ** -40, 2.0 ** -108, False),
         (2.0 ** 70, 2.0 ** 60, True), (2.0 ** 18, 2.0 ** 112, True), (2.0 ** 112, 2.0 ** 18, True),
         (2.0 ** -110, 2.0 ** 117, False), (2.0 ** 117, 2.0 ** -110, False), (2.0 ** -126, 2.0 ** 118, False),
         (2.0 ** 118, 2.0 ** -126, False)]


@pytest.mark.parametrize("sx,sw,low", PAIRS, ids=lambda v: f"{np.log2(v):.0f}" if isinstance(v, float) else None)
@pytest.mark.parametrize("rows", [5, 70, 300])
def test_scales_whose_product_leaves_fp32(rows, sx, sw, low):
    say(f"block product rows={rows} scales {sx} {sw}")
    x8, w8, x, w = _case(rows, 1, 96, 416, sx, sw, low, seed=rows)
    sd = torch.tensor([rows], dtype=torch.int32, device="cuda")
    y, _ = moe.grouped_linear_block_fwd(x8, sd, w8)
    torch.cuda.synchronize()
    ref = x @ w[0].T
    assert (ref.abs() > 2.0 ** -126).all() and (ref.abs() < 2.0 ** 127).all()
    _within(y, ref, _product_bound(x, w[0]), "y")


@pytest.mark.parametrize("rows", [5, 70, 300])
@pytest.mark.parametrize("big", [2.0 ** 70, 2.0 ** 100, 2.0 ** 114])
def test_a_block_that_sums_to_zero_adds_nothing(rows, big):
    """The first block of every row cancels exactly, with scales whose product is past fp32's range; the others
    are ordinary."""
    say(f"block product rows={rows}, zero sums at {big}")
    x8, w8, x, w = _case(rows, 1, 96, 384, 1.0, 1.0, False, seed=rows)
    codes = x8["codes"].cpu()
    codes[:, :128] = 0x38
    codes[:, 1:128:2] = 0xB8                                    # 1, -1, ..
    wc = w8["codes"].cpu()
    wc[:, :, :128] = 0x50
    xs, ws = x8["scales"].cpu(), w8["scales"].cpu()
    xs[0], ws[:, :, 0] = big, big
    y, _ = moe.grouped_linear_block_fwd({"codes": codes.cuda(), "scales": xs.cuda()},
                                        torch.tensor([rows], dtype=torch.int32, device="cuda"),
                                        {"codes": wc.cuda(), "scales": ws.cuda()})
    torch.cuda.synchronize()
    _within(y, x[:, 128:] @ w[0][:, 128:].T, _product_bound(x[:, 128:], w[0][:, 128:]), "y")


@pytest.mark.parametrize("rows", [5, 70, 300])
def test_input_gradient(rows):
    """dy of 2^-66, whose codes' scales are near 2^-74, through weights with scales near 2^-73."""
    say(f"block product backward rows={rows}, scales below fp32")
    x8, w8, _, w = _case(rows, 1, 160, 96, 1.0, 2.0 ** -73, False, seed=rows)
    g = torch.Generator().manual_seed(rows)
    dy = ((1 + torch.rand(rows, 160, generator=g)) * 2.0 ** -66).to(BF)
    dx, _ = moe.grouped_linear_block_bwd(dy.cuda(), x8, torch.tensor([rows], dtype=torch.int32, device="cuda"), w8,
                                         want_dw=False)
    torch.cuda.synchronize()
    dyq = B.rows_value(*B.quantize_rows(dy))
    ref = dyq @ w[0]
    assert (ref.abs() > 2.0 ** -126).all()
    _within(dx, ref, _product_bound(dyq, w[0].T.contiguous()), "dx")


@pytest.mark.parametrize("rows", [5, 70])
def test_zero_infinite_and_nan_scales(rows):
    """A scale of zero makes its block zeros, an infinite one an infinity where the block's sum is not zero,
    a NaN one NaN; on the rows' and on the weights' side."""
    say(f"block product rows={rows}, scales 0, inf, NaN")
    sd = torch.tensor([rows], dtype=torch.int32, device="cuda")
    for v in (0.0, float("inf"), float("nan")):
        x8, w8, x, w = _case(rows, 1, 160, 256, 1.0, 1.0, False, seed=rows)
        xs, ws = x8["scales"].clone(), w8["scales"].clone()
        xs[1, 2] = v
        ws[0, 1, 0] = v
        a, _ = moe.grouped_linear_block_fwd(x8 | {"scales": xs}, sd, w8)
        b, _ = moe.grouped_linear_block_fwd(x8, sd, w8 | {"scales": ws})
        clean, _ = moe.grouped_linear_block_fwd(x8, sd, w8)
        torch.cuda.synchronize()
        keep = torch.arange(rows) != 2
        assert torch.equal(a.cpu()[keep], clean.cpu()[keep]) and torch.equal(b[:, :128], clean[:, :128])
        got = (a[2].cpu().float(), b[:, 128:].cpu().float())
        if v == 0:
            _within(a[2:3], x[2:3, :128] @ w[0][:, :128].T, _product_bound(x[2:3, :128], w[0][:, :128]), "row")
            _within(b[:, 128:], x[:, 128:] @ w[0][128:, 128:].T, _product_bound(x[:, 128:], w[0][128:, 128:]), "weight")
        elif v == v:
            assert all(torch.isinf(t).all() and (t > 0).all() for t in got)
        else:
            assert all(t.isnan().all() for t in got)
