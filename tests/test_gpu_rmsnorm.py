"""GPU: RMS norm forward and backward against float64, element by element.

Bounds are worst-case arithmetic with u = 2^-24 (one fp32 rounding): a sum of n
terms whose longest chain of additions is c is off by at most c u sum|terms|.  A
row's chain is at most 32 values in a lane, 6 steps in a wave and 16 waves
(54 < 64 = C).  bf16 outputs add half a step, 2^-8 of the value, E4M3 codes 2^-4 of
the value or half the subnormal step, 2^-10 of the block's scale."""
import numpy as np
import pytest
import torch

import mxfp8_block_scaled_top_amd as moe
from oracle import block8 as B
from tests.helpers import need_gpu, np_, say

pytestmark = pytest.mark.gpu

U, C, TINY = 2.0 ** -24, 64, 1e-37
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
BF, F32 = torch.bfloat16, torch.float32
EPS = 1e-6


@pytest.fixture(autouse=True)
def _gpu():
    need_gpu()


def _randn(*shape, seed, dtype=F32, scale=1.0, shift=0.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale + shift).to(dtype)


def _rows(T, H, dtype, seed):
    x = _randn(T, H, seed=seed)
    x[:, :: max(1, H // 5)] *= 20.0
    return (x * (0.1 + 4 * torch.rand(T, 1, generator=torch.Generator().manual_seed(seed + 1)))).to(dtype)


def _dev(t):
    return None if t is None else t.cuda()


def _within(got, ref, bound, what):
    d = (got.double().cpu() - ref).abs()
    bad = ~(d <= bound)
    assert not bad.any(), (what, int(bad.sum()), float((d / bound.clamp_min(1e-300))[bad].max()))


def _fwd_case(T, H, xt, st, wt, res, fp8, seed, y=True):
    x = _rows(T, H, xt, seed)
    r = _rows(T, H, st, seed + 5) if res else None
    gamma = _randn(H, seed=seed + 2, dtype=wt, scale=0.3, shift=1.0) if wt else None
    got, saved = moe.moe_rmsnorm_fwd(x.cuda(), _dev(gamma), EPS, residual=_dev(r), bf16=y, fp8=fp8)
    torch.cuda.synchronize()
    h = x if r is None else (x.float() + r.float()).to(st)      # one fp32 addition, one rounding
    assert torch.equal(saved["h"].cpu(), h)
    f = B.rmsnorm_fwd(h, gamma, EPS)
    # squares u, chain C u, the mean's product and inverse 2 u, eps u: half of it, and 2 u of the root
    er = ((C + 4) / 2 + 2) * U
    _within(saved["rstd"], f["rstd"], f["rstd"] * er, "rstd")
    ey = f["y"].abs() * (er + 2.01 * U) + TINY
    if y:
        assert got.dtype == BF and got.shape == (T, H)
        _within(got, f["y"], ey + HALF[BF] * (f["y"].abs() + ey), "y")
    else:
        assert got is None
    if fp8:
        codes, scales = np_(saved["codes"]), np_(saved["scales"])
        assert codes.shape == (T, H) and scales.shape == ((H + 127) // 128, T)
        s = torch.from_numpy(scales.astype(np.float64)).T.repeat_interleave(128, 1)[:, :H]
        v = B.rows_value(codes, scales)
        _within(v, f["y"], torch.maximum(2.0 ** -4 * f["y"].abs(), 2.0 ** -10 * s) + 1.0625 * (ey + 2 * U * f["y"].abs()),
                "codes")
        top = torch.stack([b.abs().amax(1) for b in f["y"].split(128, 1)])
        want = torch.clamp(top, min=float(B.LEAST)) / 448
        _within(torch.from_numpy(scales), want, want * (er + 4 * U), "scales")


SIZES = [(1, 8), (1, 4096), (3, 40), (5, 64), (257, 96), (130, 512), (66, 520), (301, 1416), (37, 2048), (9, 2056),
         (301, 128), (67, 136), (33, 256), (7, 264), (200, 4096), (33, 4104), (17, 8192), (5, 8200), (3, 16384),
         (2, 16392), (2, 32768)]
KINDS = [(BF, BF, F32, True, True), (F32, F32, BF, False, True), (BF, F32, BF, True, True), (BF, BF, None, False, False)]


@pytest.mark.parametrize("T,H", SIZES)
@pytest.mark.parametrize("xt,st,wt,res,fp8", KINDS, ids=["bf16_res8", "f32_8", "bf16_f32stream8", "bf16"])
def test_forward(T, H, xt, st, wt, res, fp8):
    say(f"rmsnorm fwd T={T} H={H} x={xt} stream={st} w={wt} res={res} fp8={fp8}")
    _fwd_case(T, H, xt, st, wt, res, fp8, seed=H)


@pytest.mark.parametrize("T,H", [(9001, 256), (20003, 128), (2500, 2048)])
def test_forward_many_rows(T, H):
    say(f"rmsnorm fwd, more rows than workgroups at once T={T} H={H}")
    _fwd_case(T, H, BF, BF, F32, True, True, seed=5)
    _fwd_case(T, H, F32, F32, F32, True, True, seed=6, y=False)


def test_eight_bit_rows_are_the_quantizers():
    """The codes of the normed rows are those that fp8_block_quantize gives for y where
    bf16 holds y exactly: rows of +-1 and +-2 scaled by powers of two."""
    say("rmsnorm fp8 against the quantizer")
    T, H = 50, 1024
    x = torch.randint(0, 2, (T, H), generator=torch.Generator().manual_seed(1)).float() * 2 - 1     # h^2 = 1
    y, saved = moe.moe_rmsnorm_fwd(x.to(BF).cuda(), None, 0.0, fp8=True)
    codes, scales = moe.fp8_block_quantize(y)
    torch.cuda.synchronize()
    assert torch.equal(y.cpu().float(), x)
    assert torch.equal(codes, saved["codes"]) and torch.equal(scales, saved["scales"])


def _bwd_case(T, H, st, wt, res, branch, seed, want=True):
    h = _rows(T, H, st, seed)
    gamma = _randn(H, seed=seed + 2, dtype=wt, scale=0.3, shift=1.0) if wt else None
    dy, dres = _randn(T, H, seed=seed + 7, dtype=BF), (_randn(T, H, seed=seed + 8, dtype=st) if res else None)
    rstd = B.rmsnorm_fwd(h, None, EPS)["rstd"].float()
    dx, dgamma, dxb = moe.moe_rmsnorm_bwd(dy.cuda(), {"h": h.cuda(), "rstd": rstd.cuda()}, _dev(gamma),
                                          dres=_dev(dres), branch=branch, want_dgamma=want)
    torch.cuda.synchronize()
    r = B.rmsnorm_bwd(dy, h, rstd, gamma, dres)
    ga, ax = r["g"].abs(), r["xh"].abs()
    # xh rounds once; the sum: three products rounded, a chain of C additions, the division by H
    ec = (C + 6) * U * (ga * ax).mean(1, keepdim=True)
    rs = rstd.double()[:, None]
    size = ga + ax * r["c"].abs()
    e = rs * (ax * ec + 7 * U * size) * 1.01
    if res:
        e = e + 2 * U * (dres.double().abs() + rs * size)
    assert dx.dtype == st
    _within(dx, r["dx"], e + HALF[st] * (r["dx"].abs() + e) + TINY, "dx")
    if branch:
        assert dxb.dtype == BF
        _within(dxb, r["dx"], e + HALF[BF] * (r["dx"].abs() + e) + TINY, "branch")
    else:
        assert dxb is None
    if not want:
        assert dgamma is None
        return
    # rows of one thread, its wave's and workgroup's rows (32), 4 + 16 + 3 in the second kernel
    chain = (T / min(256, T) if H <= 8192 else T) + 64
    b = (chain + 4) * U * (dy.double() * r["xh"]).abs().sum(0)
    assert dgamma.dtype == (wt or F32)
    _within(dgamma, r["dgamma"], b + HALF[wt or F32] * (r["dgamma"].abs() + b) + TINY, "dgamma")


@pytest.mark.parametrize("T,H", SIZES)
@pytest.mark.parametrize("st,wt,res,branch", [(BF, F32, False, False), (F32, BF, True, True), (BF, None, True, False)],
                         ids=["bf16", "f32_res_branch", "bf16_res"])
def test_backward(T, H, st, wt, res, branch):
    say(f"rmsnorm bwd T={T} H={H} stream={st} w={wt} res={res} branch={branch}")
    _bwd_case(T, H, st, wt, res, branch, seed=H)


def test_backward_many_rows_and_without_dgamma():
    say("rmsnorm bwd, many rows")
    _bwd_case(20011, 128, BF, F32, False, False, seed=9)
    _bwd_case(20011, 256, F32, F32, True, True, seed=9)
    _bwd_case(700, 1000, F32, BF, True, False, seed=9, want=False)
    _bwd_case(70, 9000, BF, BF, False, False, seed=9, want=False)


def test_gradient_against_differences():
    """Central differences of sum(y dy) in float64 against the kernel's fp32 dx: the step 1e-4 is
    off by h^2 f''' / 6 < 1e-7, the kernel by its own bound above (< 1e-5 at these sizes)."""
    say("rmsnorm bwd against differences")
    T, H = 2, 16
    h, dy, gamma = _randn(T, H, seed=1), _randn(T, H, seed=2, dtype=BF), _randn(H, seed=3)
    _, saved = moe.moe_rmsnorm_fwd(h.cuda(), gamma.cuda(), EPS)
    dx, dgamma, _ = moe.moe_rmsnorm_bwd(dy.cuda(), saved, gamma.cuda())
    torch.cuda.synchronize()

    def f(a, g):
        return float((B.rmsnorm_fwd(a, g, EPS)["y"] * dy.double()).sum())
    for t, c in ((0, 0), (1, 5), (1, 15)):
        e = torch.zeros(T, H, dtype=torch.float64)
        e[t, c] = 1e-4
        assert abs((f(h.double() + e, gamma) - f(h.double() - e, gamma)) / 2e-4 - float(dx[t, c])) < 2e-5
    e = torch.zeros(H, dtype=torch.float64)
    e[7] = 1e-4
    assert abs((f(h, gamma.double() + e) - f(h, gamma.double() - e)) / 2e-4 - float(dgamma[7])) < 2e-5


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_non_finite_stays_in_its_row(bad):
    say(f"rmsnorm with {bad}")
    x, r = _randn(40, 320, seed=2, dtype=BF), _randn(40, 320, seed=3, dtype=BF)
    clean, s0 = moe.moe_rmsnorm_fwd(x.cuda(), None, EPS, residual=r.cuda(), fp8=True)
    x[11, 300] = bad
    y, s1 = moe.moe_rmsnorm_fwd(x.cuda(), None, EPS, residual=r.cuda(), fp8=True)
    torch.cuda.synchronize()
    keep = torch.arange(40) != 11
    assert torch.equal(y.cpu()[keep], clean.cpu()[keep])
    for k in ("codes", "rstd", "h"):
        assert torch.equal(s1[k].cpu()[keep], s0[k].cpu()[keep]), k
    assert torch.equal(s1["scales"].cpu()[:, keep], s0["scales"].cpu()[:, keep])
    v = B.rows_value(np_(s1["codes"]), np_(s1["scales"]))[11]
    assert y.cpu()[11, 300].isnan() and v[256:].isnan().all()
    if bad != bad:
        assert y.cpu()[11].isnan().all() and v.isnan().all()


def test_zero_rows_and_no_rows():
    say("rmsnorm zero rows, T=0")
    z = torch.zeros(4, 200, dtype=BF, device="cuda")
    y, saved = moe.moe_rmsnorm_fwd(z, None, EPS, fp8=True)
    dx, dgamma, _ = moe.moe_rmsnorm_bwd(torch.ones_like(z), saved)
    torch.cuda.synchronize()
    assert not y.any() and not saved["codes"].any() and (saved["scales"] == 2.0 ** -126).all() and not dgamma.any()
    assert ((dx.float() / 1000 - 1).abs() < 2.0 ** -7).all()            # rstd = eps^-1/2, dx = rstd dy
    e = torch.empty((0, 96), dtype=BF, device="cuda")
    y, saved = moe.moe_rmsnorm_fwd(e, residual=e.float(), fp8=True)
    dx, dgamma, br = moe.moe_rmsnorm_bwd(e, saved, torch.ones(96, device="cuda"), branch=True)
    torch.cuda.synchronize()
    assert y.shape == dx.shape == br.shape == (0, 96) and saved["scales"].shape == (1, 0) and not dgamma.any()


def test_writes_nothing_past_its_rows_and_works_in_place():
    """T rows of longer buffers; h over the residual, dx over dres."""
    say("rmsnorm guard rows, in place")
    T, H, G = 21, 200, 7
    L, p = moe.lib(), (lambda t: t.data_ptr())
    x, r0 = _randn(T, H, seed=6, dtype=BF).cuda(), _randn(T, H, seed=7).cuda()
    ref, saved = moe.moe_rmsnorm_fwd(x, None, EPS, residual=r0, fp8=True)
    r = torch.cat([r0, torch.full((G, H), 4.0, device="cuda")])
    y = torch.full((T + G, H), 3.0, dtype=BF, device="cuda")
    rstd = torch.full((T + G,), 5.0, device="cuda")
    codes = torch.full((T + G, H), 77, dtype=torch.uint8, device="cuda")
    scales = torch.full((2 * T + G,), 78.0, device="cuda")
    s = torch.cuda.current_stream().cuda_stream
    assert L.moe_rmsnorm_fwd(0, 1, 1, T, H, p(x), p(r), None, EPS, p(r), p(y), p(rstd), p(codes), p(scales), s) == 0
    torch.cuda.synchronize()
    assert torch.equal(r[:T], saved["h"]) and torch.equal(y[:T], ref) and torch.equal(codes[:T], saved["codes"])
    assert torch.equal(scales[:2 * T], saved["scales"].reshape(-1)) and torch.equal(rstd[:T], saved["rstd"])
    assert (r[T:] == 4).all() and (y[T:] == 3).all() and (rstd[T:] == 5).all() and (codes[T:] == 77).all()
    assert (scales[2 * T:] == 78).all()
    dres = _randn(T, H, seed=8).cuda()
    want, dg, br = moe.moe_rmsnorm_bwd(x, saved, dres=dres, branch=True)
    dx = torch.cat([dres, torch.full((G, H), 9.0, device="cuda")])
    bx = torch.full((T + G, H), 2.0, dtype=BF, device="cuda")
    dw = torch.full((H + 32,), 11.0, device="cuda")
    n = L.moe_rmsnorm_workspace_bytes(T, H)
    ws = torch.full((n + 64,), 13, dtype=torch.uint8, device="cuda")
    assert L.moe_rmsnorm_bwd(1, 1, T, H, p(x), p(r), p(rstd), None, p(dx), p(dx), p(bx), p(dw), p(ws), n, s) == 0
    torch.cuda.synchronize()
    assert torch.equal(dx[:T], want) and torch.equal(bx[:T], br) and torch.equal(dw[:H], dg)
    assert (dx[T:] == 9).all() and (bx[T:] == 2).all() and (dw[H:] == 11).all() and (ws[n:] == 13).all()


def test_offsets_past_32_bits():
    """More than 2^31 elements: the last rows are what they are by themselves."""
    say("rmsnorm with 2^31 elements")
    T, H, N = 270_000, 8192, 3000
    x = torch.empty((T, H), dtype=BF, device="cuda")
    x[:-N] = 1.0
    tail = _randn(N, H, seed=8, dtype=BF).cuda()
    x[-N:] = tail
    y, saved = moe.moe_rmsnorm_fwd(x, None, EPS, fp8=True)
    y1, s1 = moe.moe_rmsnorm_fwd(tail, None, EPS, fp8=True)
    torch.cuda.synchronize()
    assert torch.equal(y[-N:], y1) and torch.equal(saved["codes"][-N:], s1["codes"])
    assert torch.equal(saved["scales"][:, -N:], s1["scales"])
    dx = moe.moe_rmsnorm_bwd(x, saved, want_dgamma=False)[0]
    dx1 = moe.moe_rmsnorm_bwd(tail, s1, want_dgamma=False)[0]
    torch.cuda.synchronize()
    assert torch.equal(dx[-N:], dx1)


def graph_check(fn, busy):
    """Captures fn, replays it with eager work between; every replay gives the eager result."""
    ref = [t.clone() for t in fn()]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        fn()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = fn()
    for _ in range(3):
        busy()
        torch.cuda.synchronize()
        for t in got:
            t.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, ref):
            assert torch.equal(a, b)
    # the same calls on a stream of their own
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = fn()
    side.synchronize()
    for a, b in zip(other, ref):
        assert torch.equal(a, b)


def test_in_a_graph_and_on_another_stream():
    say("rmsnorm in a graph")
    T, H = 515, 1024
    x, r, gamma = _randn(T, H, seed=1, dtype=BF).cuda(), _randn(T, H, seed=2).cuda(), _randn(H, seed=3).cuda()
    dy = _randn(T, H, seed=4, dtype=BF).cuda()

    def step():
        y, saved = moe.moe_rmsnorm_fwd(x, gamma, EPS, residual=r, fp8=True)
        return [y, saved["codes"], saved["scales"], *moe.moe_rmsnorm_bwd(dy, saved, gamma, dres=r, branch=True)]

    graph_check(step, lambda: moe.moe_rmsnorm_bwd(x, moe.moe_rmsnorm_fwd(dy)[1]))


def test_binding_refusals():
    say("rmsnorm binding refusals")
    x = torch.zeros((4, 64), dtype=BF, device="cuda")
    y, saved = moe.moe_rmsnorm_fwd(x)
    f = x.float()
    for call in (
            lambda: moe.moe_rmsnorm_fwd(x.half()), lambda: moe.moe_rmsnorm_fwd(x.t()),
            lambda: moe.moe_rmsnorm_fwd(x[:, :12].contiguous()), lambda: moe.moe_rmsnorm_fwd(x, bf16=False),
            lambda: moe.moe_rmsnorm_fwd(x, torch.ones(32, device="cuda")), lambda: moe.moe_rmsnorm_fwd(x, eps=-1.0),
            lambda: moe.moe_rmsnorm_fwd(f, residual=x), lambda: moe.moe_rmsnorm_fwd(x, residual=x[:2]),
            lambda: moe.moe_rmsnorm_bwd(x, {"rstd": saved["rstd"]}), lambda: moe.moe_rmsnorm_bwd(f, saved),
            lambda: moe.moe_rmsnorm_bwd(x, saved, dres=f),
            lambda: moe.moe_rmsnorm_bwd(x, saved, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(moe.MoEError):
            call()
