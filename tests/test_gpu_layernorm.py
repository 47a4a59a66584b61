"""GPU: layer norm forward and backward against float64, element by element.

Every bound is worst-case arithmetic with u = 2^-24 (one fp32 rounding):
a fp32 sum of n terms whose longest chain of additions is c is off by at most
c u sum|terms|.  A row's chain is at most 32 values in a lane, 6 steps in a
wave and 16 waves (54 < 64 = C); the weight gradients' chain is the rows of one
workgroup, then its 4 waves and the 16-way sum over at most 512 partial rows
(32 + 16 more).  bf16 outputs add half a step, 2^-8 of the value."""
import numpy as np
import pytest
import torch

import mxfp8_block_scaled_top_amd as moe
from oracle import mx as omx
from oracle import sublayer as S
from tests.helpers import need_gpu, np_, say

pytestmark = pytest.mark.gpu

U, C, TINY = 2.0 ** -24, 64, 1e-37
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(autouse=True)
def _gpu():
    need_gpu()


def _randn(*shape, seed, dtype=F32, scale=1.0, shift=0.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale + shift).to(dtype)


def _inputs(T, H, xt, wt, seed=0):
    x = _randn(T, H, seed=seed)
    x[:, :: max(1, H // 5)] *= 20.0                                 # columns that stand out
    x = (x * (0.1 + 4 * torch.rand(T, 1, generator=torch.Generator().manual_seed(seed + 1))) + 0.5).to(xt)
    return x, _randn(H, seed=seed + 2, dtype=wt, scale=0.3, shift=1.0), _randn(H, seed=seed + 3, dtype=wt)


def _within(got, ref, bound, what):
    d = (got.double().cpu() - ref).abs()
    bad = ~(d <= bound)
    assert not bad.any(), (what, int(bad.sum()), float((d / bound.clamp_min(1e-300))[bad].max()))


def _xh_error(x, f):
    """Bound of |xh - xh64| for the forward's fp32 arithmetic: the mean is off
    by C u mean|x|, the difference rounds once, the sum of squares is off by
    C u of itself plus what the mean's error adds (its square, the linear term
    cancels), and rstd takes half of that, the division and root 4 u."""
    r = f["rstd"][:, None]
    dm = C * U * x.double().abs().mean(1, keepdim=True)
    dr = (C + 8) * U + (dm * r) ** 2 + 2 * U * (x.double().abs().amax(1, keepdim=True) * r)
    return r * (dm + U * (x.double().abs() + dm)) + f["xh"].abs() * dr + TINY


def _check_ckpt(saved, xh, err):
    codes, scales = np_(saved["xhat_codes"]), np_(saved["xhat_scales"])
    v = torch.from_numpy(omx.dequantize_rows(codes, scales)).double()
    X = torch.from_numpy(2.0 ** (scales.astype(np.float64) - 127)).repeat_interleave(32, 1)
    # half a step of E4M3: 2^-4 of a value, at least half the subnormal step 2^-9 X
    assert ((v - xh).abs() <= torch.maximum(2.0 ** -4 * xh.abs(), 2.0 ** -10 * X) + 1.0625 * err).all()
    top = xh.abs().reshape(*scales.shape, 32).amax(2)
    slack = err.reshape(*scales.shape, 32).amax(2)
    Xb = torch.from_numpy(2.0 ** (scales.astype(np.float64) - 127))
    live = torch.from_numpy(scales > 0)
    assert (top <= 448 * Xb + slack).all() and (top >= 224 * Xb - slack)[live].all()


def _fwd_case(T, H, xt, wt, ckpt, seed=0, eps=1e-5, affine=True):
    x, gamma, beta = _inputs(T, H, xt, wt, seed)
    if not affine:
        gamma = beta = None
    dev = lambda t: None if t is None else t.cuda()                  # noqa: E731
    y, saved = moe.moe_layernorm_fwd(dev(x), dev(gamma), dev(beta), eps, checkpoint=ckpt)
    torch.cuda.synchronize()
    f = S.layernorm_fwd(x, gamma, beta, eps)
    err = _xh_error(x, f)
    ga = torch.ones(H, dtype=torch.float64) if gamma is None else gamma.double().abs()
    be = torch.zeros(H, dtype=torch.float64) if beta is None else beta.double().abs()
    ey = ga * err * 1.01 + 2 * U * (ga * f["xh"].abs() + be)
    assert y.dtype == BF and y.shape == (T, H)
    _within(y, f["y"], ey + HALF[BF] * (f["y"].abs() + ey) + TINY, "y")
    xa = x.double().abs()
    _within(saved["mean"], f["mean"], (C + 2) * U * xa.mean(1) + TINY, "mean")
    dm = C * U * xa.mean(1)
    _within(saved["rstd"], f["rstd"],
            f["rstd"] * ((C + 10) * U + (dm * f["rstd"]) ** 2 + 2 * U * xa.amax(1) * f["rstd"]), "rstd")
    if ckpt:
        _check_ckpt(saved, f["xh"], err)


SIZES = [(1, 8), (1, 4096), (3, 40), (5, 64), (257, 96), (130, 512), (66, 520), (1001, 1416), (37, 2048),
         (9, 2056), (301, 128), (67, 136), (33, 256), (7, 264), (300, 4096), (33, 4104), (17, 8192), (5, 8200), (3, 16384), (2, 16392), (2, 32768)]


@pytest.mark.parametrize("T,H", SIZES)
@pytest.mark.parametrize("xt,wt", [(BF, F32), (F32, BF)], ids=["bf16", "f32"])
def test_forward(T, H, xt, wt):
    say(f"layernorm fwd T={T} H={H} x={xt} w={wt}")
    _fwd_case(T, H, xt, wt, ckpt=H % 32 == 0, seed=H)


def test_forward_without_weights():
    say("layernorm fwd without gamma and beta")
    _fwd_case(19, 384, BF, F32, True, affine=False)


def test_forward_many_rows():
    say("layernorm fwd, more rows than workgroups at once")
    _fwd_case(9001, 256, F32, F32, True, seed=5)
    _fwd_case(20003, 128, BF, F32, True, seed=6)


def _xh32(x, mean, rstd):
    return ((x.float() - mean[:, None]) * rstd[:, None]).double()


def _bwd_case(T, H, xt, wt, ckpt, res, seed=0, affine=True, want=(True, True)):
    x, gamma, _ = _inputs(T, H, xt, wt, seed)
    if not affine:
        gamma, wt = None, F32
    dy, dres = _randn(T, H, seed=seed + 7, dtype=BF), (_randn(T, H, seed=seed + 8, dtype=xt) if res else None)
    f = S.layernorm_fwd(x)
    mean, rstd = f["mean"].float(), f["rstd"].float()
    saved = {"mean": mean.cuda(), "rstd": rstd.cuda()}
    if ckpt:
        codes, scales = omx.quantize_rows((f["xh"]).float())
        saved |= {"xhat_codes": torch.from_numpy(codes).cuda(), "xhat_scales": torch.from_numpy(scales).cuda()}
        xh = torch.from_numpy(omx.dequantize_rows(codes, scales)).double()
        exh = torch.zeros_like(xh)
    else:
        # xh from the given fp32 statistics: the difference and the product round
        xh = (x.double() - mean.double()[:, None]) * rstd.double()[:, None]
        exh = 2.01 * U * xh.abs()
    dev = lambda t: None if t is None else t.cuda()                  # noqa: E731
    dx, dgamma, dbeta = moe.moe_layernorm_bwd(dy.cuda(), saved, dev(gamma), x=None if ckpt else x.cuda(),
                                              dres=dev(dres), dx_dtype=xt, want_dgamma=want[0],
                                              want_dbeta=want[1])
    torch.cuda.synchronize()
    r = S.layernorm_bwd(dy, xh, rstd, gamma, dres)
    ga, ax = r["g"].abs(), xh.abs()
    # c1, c2: products rounded, a chain of C additions, the division by H
    e1 = (C + 3) * U * ga.mean(1, keepdim=True)
    e2 = (C + 4) * U * (ga * ax).mean(1, keepdim=True) + (ga * exh).mean(1, keepdim=True) * 1.01
    rs = rstd.double()[:, None]
    size = ga + r["c1"].abs() + ax * r["c2"].abs()
    e = rs * (e1 + ax * e2 + exh * r["c2"].abs() + 6 * U * size) * 1.01
    if res:
        e = e + 2 * U * (dres.double().abs() + rs * size)
    assert dx.dtype == xt
    _within(dx, r["dx"], e + HALF[xt] * (r["dx"].abs() + e) + TINY, "dx")
    chain = T / min(512, T) + 4 + 64
    for got, ref, mag, err, w in ((dgamma, r["dgamma"], (dy.double() * xh).abs().sum(0),
                                   (dy.double().abs() * exh).sum(0), want[0]),
                                  (dbeta, r["dbeta"], dy.double().abs().sum(0), 0.0, want[1])):
        if not w:
            assert got is None
            continue
        assert got.dtype == wt
        b = (chain + 2) * U * mag + 1.01 * err
        _within(got, ref, b + HALF[wt] * (ref.abs() + b) + TINY, "dw")


@pytest.mark.parametrize("T,H", SIZES)
@pytest.mark.parametrize("xt,wt,res", [(BF, F32, False), (F32, BF, True)], ids=["bf16", "f32_res"])
def test_backward(T, H, xt, wt, res):
    say(f"layernorm bwd T={T} H={H} x={xt} w={wt} res={res}")
    _bwd_case(T, H, xt, wt, False, res, seed=H)


@pytest.mark.parametrize("T,H", [s for s in SIZES if s[1] % 32 == 0])
@pytest.mark.parametrize("xt,wt,res", [(BF, BF, True), (F32, F32, False)], ids=["bf16_res", "f32"])
def test_backward_from_checkpoint(T, H, xt, wt, res):
    say(f"layernorm bwd from 8 bits T={T} H={H} x={xt} w={wt} res={res}")
    _bwd_case(T, H, xt, wt, True, res, seed=H)


@pytest.mark.parametrize("want", [(False, False), (True, False), (False, True)])
def test_backward_wanted_gradients(want):
    say(f"layernorm bwd want={want}")
    _bwd_case(70, 192, BF, F32, True, False, affine=want[0], want=want)


def test_backward_many_rows():
    say("layernorm bwd, many rows")
    _bwd_case(20011, 128, BF, F32, False, False, seed=9)
    _bwd_case(20011, 256, BF, F32, True, False, seed=9)


def test_constant_rows_and_zero_rows():
    """Variance 0: xh is 0 (eps keeps rstd finite) and its blocks are code 0, scale 0."""
    say("layernorm constant rows")
    T, H = 6, 256
    x = torch.full((T, H), 0.75, dtype=BF)
    x[3:] = 0
    y, saved = moe.moe_layernorm_fwd(x.cuda(), checkpoint=True)
    torch.cuda.synchronize()
    assert not y.any() and not saved["xhat_codes"].any() and not saved["xhat_scales"].any()
    dy = _randn(T, H, seed=1, dtype=BF)
    dx, dgamma, _ = moe.moe_layernorm_bwd(dy.cuda(), saved)
    torch.cuda.synchronize()
    r = S.layernorm_bwd(dy, torch.zeros(T, H), saved["rstd"].cpu())
    assert not dgamma.any()
    _within(dx, r["dx"], 2.0 ** -8 * r["dx"].abs() + 316.3 * (C + 8) * U * (dy.double().abs() + 1), "dx")


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_non_finite_stays_in_its_row(bad):
    say(f"layernorm with {bad}")
    x = _randn(40, 320, seed=2, dtype=BF)
    clean, s0 = moe.moe_layernorm_fwd(x.cuda())
    x[11, 300] = bad
    y, s1 = moe.moe_layernorm_fwd(x.cuda())
    torch.cuda.synchronize()
    keep = torch.arange(40) != 11
    assert torch.equal(y.cpu()[keep], clean.cpu()[keep])
    assert torch.equal(s1["rstd"].cpu()[keep], s0["rstd"].cpu()[keep])
    assert y.cpu()[11].isnan().all() and s1["rstd"].cpu()[11].isnan()


@pytest.mark.parametrize("big", [1e4, 3e4])
def test_large_mean_does_not_cancel(big):
    """Rows whose mean is far above their spread: the variance is summed around the mean."""
    say(f"layernorm with mean {big}")
    T, H = 8, 1024
    x = _randn(T, H, seed=3, shift=big)
    y, saved = moe.moe_layernorm_fwd(x.cuda())
    torch.cuda.synchronize()
    f = S.layernorm_fwd(x)
    err = _xh_error(x, f)
    _within(y, f["y"], err * 1.01 + 2.0 ** -8 * (f["y"].abs() + err), "y")
    assert ((saved["rstd"].double().cpu() / f["rstd"] - 1).abs() < 0.02).all()


def test_no_rows():
    say("layernorm T=0")
    e = torch.empty((0, 96), dtype=BF, device="cuda")
    y, saved = moe.moe_layernorm_fwd(e, checkpoint=True)
    dx, dgamma, dbeta = moe.moe_layernorm_bwd(e, saved, torch.ones(96, device="cuda"))
    torch.cuda.synchronize()
    assert y.shape == (0, 96) and dx.shape == (0, 96)
    assert not dgamma.any() and not dbeta.any()


def test_same_bits_every_time_and_residual_in_place():
    say("layernorm bwd twice, dres in place")
    T, H = 3001, 640
    x, gamma, _ = _inputs(T, H, BF, F32)
    dy, dres = _randn(T, H, seed=4, dtype=BF).cuda(), _randn(T, H, seed=5, dtype=BF).cuda()
    _, saved = moe.moe_layernorm_fwd(x.cuda(), gamma.cuda(), checkpoint=True)
    a = moe.moe_layernorm_bwd(dy, saved, gamma.cuda(), dres=dres)
    b = moe.moe_layernorm_bwd(dy, saved, gamma.cuda(), dres=dres)
    torch.cuda.synchronize()
    for p, q in zip(a, b):
        assert torch.equal(p, q)
    # the C entry point with dx = dres
    L, p = moe.lib(), (lambda t: t.data_ptr())
    g = gamma.cuda()
    assert L.moe_layernorm_bwd(0, 1, T, H, p(dy), None, None, p(saved["rstd"]), p(saved["xhat_codes"]),
                               p(saved["xhat_scales"]), p(g), p(dres), p(dres), None, None, None, 0,
                               torch.cuda.current_stream().cuda_stream) == 0
    torch.cuda.synchronize()
    assert torch.equal(dres, a[0])


def test_writes_nothing_past_its_rows():
    """T rows of longer buffers: what lies behind stays as it was."""
    say("layernorm guard rows")
    T, H, G = 21, 160, 7
    x = _randn(T, H, seed=6, dtype=BF).cuda()
    L, p = moe.lib(), (lambda t: t.data_ptr())
    y = torch.full((T + G, H), 3.0, dtype=BF, device="cuda")
    st = torch.full((2, T + G), 5.0, device="cuda")
    codes = torch.full((T + G, H), 77, dtype=torch.uint8, device="cuda")
    scales = torch.full((T + G, H // 32), 78, dtype=torch.uint8, device="cuda")
    s = torch.cuda.current_stream().cuda_stream
    assert L.moe_layernorm_fwd(0, 1, T, H, p(x), None, None, 1e-5, p(y), p(st[0]), p(st[1]), p(codes),
                               p(scales), s) == 0
    dx = torch.full((T + G, H), 9.0, device="cuda")
    dw = torch.full((2, H + 32), 11.0, device="cuda")
    n = L.moe_layernorm_workspace_bytes(T, H)
    ws = torch.full((n + 64,), 13, dtype=torch.uint8, device="cuda")
    assert L.moe_layernorm_bwd(1, 1, T, H, p(x), None, None, p(st[1]), p(codes), p(scales), None, None,
                               p(dx), p(dw[0]), p(dw[1]), p(ws), n, s) == 0
    torch.cuda.synchronize()
    assert (y[T:] == 3).all() and (st[:, T:] == 5).all() and (codes[T:] == 77).all()
    assert (scales[T:] == 78).all() and (dx[T:] == 9).all() and (dw[:, H:] == 11).all()
    assert (ws[n:] == 13).all() and not (dx[:T] == 9).any()


def test_offsets_past_32_bits():
    """More than 2^31 elements: the last rows are what they are by themselves."""
    say("layernorm with 2^31 elements")
    T, H = 270_000, 8192
    x = torch.empty((T, H), dtype=BF, device="cuda")
    x[:-3000] = 1.0
    tail = _randn(3000, H, seed=8, dtype=BF).cuda()
    x[-3000:] = tail
    y, saved = moe.moe_layernorm_fwd(x, checkpoint=True)
    y1, s1 = moe.moe_layernorm_fwd(tail, checkpoint=True)
    torch.cuda.synchronize()
    assert torch.equal(y[-3000:], y1)
    for k in s1:
        assert torch.equal(saved[k][-3000:], s1[k]), k
    dx = moe.moe_layernorm_bwd(x, saved, want_dgamma=False, want_dbeta=False)[0]
    dx1 = moe.moe_layernorm_bwd(tail, s1, want_dgamma=False, want_dbeta=False)[0]
    torch.cuda.synchronize()
    assert torch.equal(dx[-3000:], dx1)


def _graph_check(fn, outs, busy):
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


def test_in_a_graph_and_on_another_stream():
    say("layernorm in a graph")
    T, H = 515, 1024
    x, gamma, beta = (t.cuda() for t in _inputs(T, H, BF, F32))
    dy = _randn(T, H, seed=4, dtype=BF).cuda()

    def step():
        y, saved = moe.moe_layernorm_fwd(x, gamma, beta, checkpoint=True)
        return [y, saved["xhat_codes"], *moe.moe_layernorm_bwd(dy, saved, gamma)]

    _graph_check(step, None, lambda: moe.moe_layernorm_bwd(x, moe.moe_layernorm_fwd(dy)[1], x=dy))
    ref = step()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        other = step()
    s.synchronize()
    for a, b in zip(ref, other):
        assert torch.equal(a, b)


def test_checkpoint_takes_the_place_of_x():
    """With a checkpoint x only gives dx its type."""
    say("layernorm bwd with both")
    x = _randn(20, 96, seed=1).cuda()
    dy = _randn(20, 96, seed=2, dtype=BF).cuda()
    _, saved = moe.moe_layernorm_fwd(x, checkpoint=True)
    a = moe.moe_layernorm_bwd(dy, saved, x=x)
    b = moe.moe_layernorm_bwd(dy, saved, dx_dtype=F32)
    torch.cuda.synchronize()
    assert a[0].dtype == F32 and torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_binding_refusals():
    say("layernorm binding refusals")
    x = torch.zeros((4, 64), dtype=BF, device="cuda")
    y, saved = moe.moe_layernorm_fwd(x, checkpoint=True)
    for call in (
            lambda: moe.moe_layernorm_fwd(x.half()), lambda: moe.moe_layernorm_fwd(x.t()),
            lambda: moe.moe_layernorm_fwd(x[:, :12].contiguous()),
            lambda: moe.moe_layernorm_fwd(x[:, :40].contiguous(), checkpoint=True),
            lambda: moe.moe_layernorm_fwd(x, torch.ones(32, device="cuda")),
            lambda: moe.moe_layernorm_fwd(x, torch.ones(64, device="cuda"), torch.ones(64, device="cuda", dtype=BF)),
            lambda: moe.moe_layernorm_fwd(x, eps=-1.0),
            lambda: moe.moe_layernorm_bwd(x, {"rstd": saved["rstd"], "mean": saved["mean"]}),
            lambda: moe.moe_layernorm_bwd(x, saved | {"xhat_codes": saved["xhat_codes"][:2]}),
            lambda: moe.moe_layernorm_bwd(x, saved, dres=x.float(), dx_dtype=BF),
            lambda: moe.moe_layernorm_bwd(x, {"mean": saved["mean"], "rstd": saved["rstd"]}, x=x, dx_dtype=F32),
            lambda: moe.moe_layernorm_bwd(x, saved, dx_dtype=torch.float16),
            lambda: moe.moe_layernorm_bwd(x, saved, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(moe.MoEError):
            call()
