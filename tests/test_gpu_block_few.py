"""GPU: block products at up to 8 rows per expert on average whose rows are not spread evenly: an expert takes
its rows 16 at a time, one pass after the other.  Bounds as in test_gpu_block_linear."""
import pytest
import torch

import mxfp8_block_scaled_top_amd as moe
from oracle import block8 as B
from tests.helpers import need_gpu, say
from tests.test_gpu_block_linear import BF, H8, U, _check, _check_fwd, _problem, _product_bound, _randn

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    need_gpu()


# (split, N, K): blocks of K for one, some and all of a workgroup's eight waves, and for two rounds of them
CASES = [([6], 32, 32), ([8], 96, 416), ([16, 0], 160, 128), ([17] + [0] * 7, 288, 1120), ([33, 1, 0, 0, 0, 16, 0, 0], 96, 1408),
         ([0, 0, 0, 64, 0, 0, 0, 0], 544, 256), ([100] + [0] * 15, 64, 2080), ([15, 17, 16, 0, 31, 32, 33] + [0] * 20, 96, 192),
         ([0] * 60 + [497, 3, 0, 12], 96, 416), ([2, 48, 0, 14] + [0] * 4, 2080, 96)]


@pytest.mark.parametrize("split,N,K", CASES)
@pytest.mark.parametrize("gather", [False, True], ids=["rows", "gather"])
def test_uneven_few_rows(split, N, K, gather):
    rows = sum(split)
    say(f"few rows {rows} over {len(split)}, most {max(split)}, N={N} K={K} gather={gather}")
    assert rows <= 8 * len(split)
    p = _problem(split, len(split), N, K, seed=N + 3 * K, tokens=rows // 2 + 1 if gather else 0)
    dy = _randn(rows, N, seed=5)
    y, _ = moe.grouped_linear_block_fwd(p["x8"], p["sd"], p["w8"], src_token=p["src"])
    z, _ = moe.grouped_linear_block_fwd(p["x8"], p["sd"], p["w8"], src_token=p["src"])
    dx, dw = moe.grouped_linear_block_bwd(dy.cuda(), p["x8"], p["sd"], p["w8"], src_token=p["src"])
    torch.cuda.synchronize()
    _check_fwd(p, y)
    assert torch.equal(y, z)
    dyq = B.rows_value(*B.quantize_rows(dy))
    rx, rw = B.linear_bwd(dy, dyq, p["x"], p["w"], split)
    at = 0
    for e, n in enumerate(split):
        _check(dx[at:at + n], rx[at:at + n], _product_bound(dyq[at:at + n], p["w"][e].T.contiguous()), f"dx {e}")
        mag = dy[at:at + n].double().abs().T @ p["x"][at:at + n].abs()
        _check(dw[e], rw[e], (H8 + (n + 8) * U) * mag, f"dw {e}")
        at += n


def test_the_same_rows_on_one_expert_and_as_tiles():
    """40 rows on one of eight experts (in passes) and the same with 100 more on another (in tiles): each output
    has the same products, and both are what the formula says."""
    say("few rows against tiles")
    N, K, E = 160, 672, 8
    p = _problem([0, 40, 0, 100, 0, 0, 0, 0], E, N, K, seed=2)
    few = {"codes": p["x8"]["codes"][:40].contiguous(), "scales": p["x8"]["scales"][:, :40].contiguous()}
    y, _ = moe.grouped_linear_block_fwd(p["x8"], p["sd"], p["w8"])
    sd = torch.tensor([0, 40] + [0] * 6, dtype=torch.int32, device="cuda")
    z, _ = moe.grouped_linear_block_fwd(few, sd, p["w8"])
    torch.cuda.synchronize()
    _check_fwd(p, y)
    bound = _product_bound(p["x"][:40], p["w"][1])
    _check(z, p["x"][:40] @ p["w"][1].T, bound, "passes")


@pytest.mark.parametrize("N,K", [(96, 160), (288, 1120)])
def test_rows_behind_the_last_expert_stay(N, K):
    say(f"few rows, guard rows, N={N} K={K}")
    split = [0, 21, 0, 2] + [0] * 12
    p = _problem(split, 16, N, K, seed=4, extra=30)
    assert p["rows"] <= 8 * 16
    L, q = moe.lib(), (lambda t: t.data_ptr())
    s = torch.cuda.current_stream().cuda_stream
    ws = moe._ptr_array(list(p["w8"]["scales"]))
    y = torch.full((p["rows"] + 9, N), 3.0, dtype=BF, device="cuda")
    assert L.grouped_linear_block_fwd(16, N, K, p["rows"], q(p["x8"]["codes"]), q(p["x8"]["scales"]), p["rows"], None,
                                      q(p["sd"]), moe._ptr_array(list(p["w8"]["codes"])), ws, q(y), s) == 0
    dx = torch.full((p["rows"] + 9, K), 4.0, dtype=BF, device="cuda")
    n = moe.moe_workspace_bytes(moe.MOE_OP_LINEAR_BLOCK_BWD, p["rows"], K, N, 16, 1, 0)
    wk = torch.full((n + 64,), 6, dtype=torch.uint8, device="cuda")
    dy = _randn(p["rows"], N, seed=6)
    dyd = dy.cuda()
    assert L.grouped_linear_block_bwd(16, N, K, p["rows"], q(dyd), q(p["x8"]["codes"]), q(p["x8"]["scales"]), p["rows"],
                                      None, q(p["sd"]), moe._ptr_array(list(p["w8"]["codes_t"])), ws, q(dx), None, q(wk), n,
                                      s) == 0
    torch.cuda.synchronize()
    _check_fwd(p, y)
    assert (y[23:] == 3).all() and (dx[23:] == 4).all() and (wk[n:] == 6).all()
    dyq = B.rows_value(*B.quantize_rows(dy))
    _check(dx[:21], dyq[:21] @ p["w"][1], _product_bound(dyq[:21], p["w"][1].T.contiguous()), "dx")


@pytest.mark.parametrize("split", [[-5, 20, 30], [50, 50, 50], [0, 0, 0], [2 ** 31 - 1, 2 ** 31 - 1, 5], [40, -2 ** 31, 1]])
def test_bad_sizes_stay_inside(split):
    """60 rows for 16 experts: negative sizes count as 0, and what passes the rows is cut."""
    say(f"few rows, sizes {split}")
    split = split + [0] * 13
    p = _problem([20, 30, 10] + [0] * 13, 16, 96, 160, seed=7)
    sd = torch.tensor(split, dtype=torch.int64).to(torch.int32).cuda()
    buf = torch.full((p["rows"] + 40, 96), 3.0, dtype=BF, device="cuda")
    L, q = moe.lib(), (lambda t: t.data_ptr())
    wc, ws = moe._ptr_array(list(p["w8"]["codes"])), moe._ptr_array(list(p["w8"]["scales"]))
    assert L.grouped_linear_block_fwd(16, 96, 160, p["rows"], q(p["x8"]["codes"]), q(p["x8"]["scales"]), p["rows"], None,
                                      q(sd), wc, ws, q(buf), torch.cuda.current_stream().cuda_stream) == 0
    torch.cuda.synchronize()
    cut, left = [], p["rows"]
    for n in split:
        cut.append(min(max(n, 0), left))
        left -= cut[-1]
    assert (buf[sum(cut):] == 3).all()
    at = 0
    for e, n in enumerate(cut):
        a = p["x"][at:at + n]
        _check(buf[at:at + n], a @ p["w"][e].T, _product_bound(a, p["w"][e]), "cut")
        at += n


@pytest.mark.parametrize("bad", [-1, 31, 2 ** 31 - 1, -2 ** 31])
def test_tokens_out_of_range_are_rows_of_zeros(bad):
    say(f"few rows, src_token {bad}")
    p = _problem([0, 40, 0, 0, 1, 0, 0, 2], 8, 96, 160, seed=9, tokens=31)
    clean, _ = moe.grouped_linear_block_fwd(p["x8"], p["sd"], p["w8"], src_token=p["src"])
    src = p["src"].clone()
    hit = torch.tensor([0, 17, 39, 42])
    src[hit.cuda()] = bad
    y, _ = moe.grouped_linear_block_fwd(p["x8"], p["sd"], p["w8"], src_token=src)
    torch.cuda.synchronize()
    keep = torch.ones(43, dtype=torch.bool)
    keep[hit] = False
    assert not y.cpu()[~keep].any() and torch.equal(y.cpu()[keep], clean.cpu()[keep])


def test_nan_stays_in_its_row_past_the_first_pass():
    say("few rows, NaN in a later pass")
    p = _problem([0, 50, 0, 0, 0, 0, 0, 0], 8, 96, 1184, seed=10)
    clean, _ = moe.grouped_linear_block_fwd(p["x8"], p["sd"], p["w8"])
    codes = p["x8"]["codes"].clone()
    codes[21, 1150] = 0x7F
    y, _ = moe.grouped_linear_block_fwd(p["x8"] | {"codes": codes}, p["sd"], p["w8"])
    torch.cuda.synchronize()
    keep = torch.arange(50) != 21
    assert y[21].isnan().all() and torch.equal(y.cpu()[keep], clean.cpu()[keep])
    assert not clean.isnan().any()
