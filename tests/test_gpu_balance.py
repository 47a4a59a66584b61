"""GPU: balance loss, counts and the logits' gradient against float64.

Bounds with u = 2^-24.  A probability: the difference from the row's top rounds (u of the
range R), expf 2 u, a sum of at most 4 in a lane and 6 steps (12 u), the inverse and the
product 2 u: (2 R + 32) u of itself covers numerator and denominator."""
import pytest
import torch

import mxfp8_block_scaled_top_amd as moe
from oracle import block8 as B
from tests.helpers import need_gpu, say
from tests.test_gpu_rmsnorm import graph_check

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(autouse=True)
def _gpu():
    need_gpu()


def _case(T, E, k, seed, masked=False, add=False, skew=0.7):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, E, generator=g) * 1.5 + skew * torch.randn(E, generator=g)
    topk = torch.topk(x, k, 1).indices.int()
    mask = (torch.rand(T, generator=g) < 0.7) if masked else None
    d0 = torch.randn(T, E, generator=g) * 1e-3 if add else None
    return x, topk, mask, d0


def _within(got, ref, bound, what):
    d = (got.double().cpu() - ref).abs()
    assert (d <= bound).all(), (what, float((d / bound.clamp_min(1e-300)).max()))


def _check(x, topk, mask, d0, coef, z, dloss=None):
    T, E = x.shape
    dev = lambda t: None if t is None else t.cuda()                 # noqa: E731
    loss, saved = moe.moe_balance_fwd(x.cuda(), topk.cuda(), dev(mask), coef, z)
    up = None if dloss is None else torch.tensor([dloss], device="cuda")
    d = moe.moe_balance_bwd(x.cuda(), saved, dev(mask), up, dlogits=dev(d0))
    torch.cuda.synchronize()
    r = B.balance(x, topk, mask, coef, z, 1.0 if dloss is None else dloss)
    assert torch.equal(saved["counts"].cpu(), r["counts"]) and int(saved["tokens"]) == r["tokens"]
    n = max(1, r["tokens"])
    fin = x.double().masked_fill(~x.isfinite(), 0.0)
    R = (fin.amax(1, keepdim=True) - fin.amin(1, keepdim=True)) if T else torch.zeros(0, 1).double()
    ep = (2 * R + 32) * U                                            # relative, per token
    el = (R.squeeze(1) + 24) * U + 4 * U * (r["lse"].abs() + fin.abs().amax(1)) if T else torch.zeros(0).double()
    chain = T / 1024 + 1 + 12       # tokens of one lane (256 workgroups of at least 4 at once), wave, workgroup
    eP = (r["p"] * (ep + chain * U)).sum(0) / n + 2 * U * r["mean_prob"]
    _within(saved["mean_prob"], r["mean_prob"], eP + 1e-37, "mean_prob")
    eb = abs(coef) * E * (r["f"] * (eP + U * r["mean_prob"])).sum() + 4 * U * r["balance"].abs()
    l2 = r["lse"] * r["lse"]
    ez = abs(z) / n * (2.1 * r["lse"].abs() * el + (chain + 3) * U * l2).sum() + 3 * U * r["z"].abs()
    _within(saved["losses"][1], r["balance"], eb + 1e-37, "balance")
    _within(saved["losses"][2], r["z"], ez + 1e-37, "z")
    _within(loss, r["loss"], eb + ez + U * r["loss"].abs() + 1e-37, "loss")
    up = abs(dloss) if dloss is not None else 1.0
    s = (r["p"] * r["f"]).sum(1, keepdim=True)
    cb, cz = up * abs(coef) * E / n, up * 2 * abs(z) / n
    mag = cb * (r["f"] + s) + cz * r["lse"].abs()[:, None]
    e = r["p"] * (cb * (s * (ep + 14 * U) + 4 * U * r["f"]) + cz * el[:, None] + (ep + 12 * U) * mag)
    ref = r["dlogits"] if d0 is None else r["dlogits"] + d0.double()
    if d0 is not None:
        e = e + U * (ref.abs() + d0.double().abs())
    _within(d, ref, e * 1.01 + 1e-37, "dlogits")
    if mask is not None and d0 is not None:
        assert torch.equal(d.cpu()[~mask.bool()], d0[~mask.bool()])


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 64, 8), (2, 2, 1), (7, 3, 2), (64, 4, 4), (256, 4, 2), (300, 5, 5),
                                   (513, 8, 2), (129, 12, 3), (77, 16, 2), (250, 17, 4), (999, 32, 6), (40, 33, 1),
                                   (2500, 60, 8), (1500, 63, 2), (4099, 64, 8), (70001, 61, 3), (300, 1, 1)])
@pytest.mark.parametrize("masked,add", [(False, False), (True, True)], ids=["plain", "mask_add"])
def test_losses_and_gradient(T, E, k, masked, add):
    say(f"balance T={T} E={E} k={k} mask={masked} add={add}")
    x, topk, mask, d0 = _case(T, E, k, seed=T + E, masked=masked, add=add)
    _check(x, topk, mask, d0, 0.01, 0.001, None if add else 2.5)


def test_offsets_past_32_bits():
    """2.2 billion logits, zeros but for the last rows; every token picks expert 0, so f = (1, 0, ..).  Probabilities
    carry some 8 roundings (exponential, sum, quotient), the products after them 4 more: 16 u of the terms' sizes."""
    T, E, n = 34_000_000, 64, 500
    say(f"balance {T} x {E}")
    logits = torch.zeros((T, E), device="cuda")
    x = torch.randn(n, E, generator=torch.Generator().manual_seed(5))
    logits[-n:] = x.cuda()
    loss, saved = moe.moe_balance_fwd(logits, torch.zeros((T, 1), dtype=torch.int32, device="cuda"), balance_coef=1.0)
    d = moe.moe_balance_bwd(logits, saved)
    torch.cuda.synchronize()
    p = x.double().softmax(-1)
    P0 = (p[:, 0].sum() + (T - n) / 64) / T
    assert saved["counts"].tolist() == [T] + [0] * 63 and int(saved["tokens"]) == T
    assert abs(float(loss) - float(64 * P0)) <= 64 * 2.0 ** -24
    f = torch.zeros(E).double()
    f[0] = 1
    want = 64 / T * p * (f - p[:, :1])
    lim = 16 * 2.0 ** -24 * 64 / T * p * (f + p[:, :1])
    assert ((d[-n:].cpu().double() - want).abs() <= lim).all()
    first = 64 / T / 64 * (f - 1 / 64)
    assert ((d[[0, 1, T // 2]].cpu().double() - first).abs() <= 16 * 2.0 ** -24 * first.abs()).all()


def test_one_loss_alone_and_large_coefficients():
    say("balance: one loss at a time")
    c = _case(333, 10, 3, seed=1)
    _check(*c, 1.0, 0.0)
    _check(*c, 0.0, 1.0)
    _check(*c, -3.0, 0.0)


def test_no_token_counts():
    say("balance: nothing counts")
    x, topk, _, d0 = _case(50, 6, 2, seed=2, add=True)
    x[3] = float("nan")                                              # not read
    mask = torch.zeros(50, dtype=torch.uint8)
    loss, saved = moe.moe_balance_fwd(x.cuda(), topk.cuda(), mask.cuda(), 0.1, 0.1)
    d = moe.moe_balance_bwd(x.cuda(), saved, mask.cuda(), dlogits=d0.cuda())
    torch.cuda.synchronize()
    assert float(loss) == 0 and not saved["counts"].any() and int(saved["tokens"]) == 0
    assert not saved["mean_prob"].any() and torch.equal(d.cpu(), d0)
    e = torch.empty(0, 6, device="cuda")
    loss, saved = moe.moe_balance_fwd(e, torch.empty(0, 2, dtype=torch.int32, device="cuda"))
    assert moe.moe_balance_bwd(e, saved).shape == (0, 6)
    assert float(loss) == 0 and not saved["counts"].any()


def test_masked_experts_and_empty_rows():
    """-infinity for experts that a token may not take, also for all of them."""
    say("balance: -inf logits")
    x, topk, mask, _ = _case(200, 8, 2, seed=3, masked=True)
    x[:, 5] = -float("inf")
    x[::7, :4] = -float("inf")
    x[11] = -float("inf")
    x[12] = torch.finfo(torch.float32).min
    _check(x, topk, mask, None, 0.02, 0.0)
    loss, saved = moe.moe_balance_fwd(x.cuda(), topk.cuda(), None, 0.02, 0.0)
    d = moe.moe_balance_bwd(x.cuda(), saved)
    torch.cuda.synchronize()
    # (row 12 has eight equal logits, expert 5's among them: p = 1/8 there)
    keep = torch.arange(200) != 12
    assert loss.isfinite() and d.isfinite().all() and not d[11].any() and not d.cpu()[keep, 5].any()


def test_nan_shows_and_stays_in_its_row():
    say("balance: NaN")
    x, topk, _, _ = _case(70, 8, 2, seed=4)
    x[20, 3] = float("nan")
    loss, saved = moe.moe_balance_fwd(x.cuda(), topk.cuda(), None, 0.02, 0.0)
    d = moe.moe_balance_bwd(x.cuda(), saved).cpu()
    assert loss.isnan() and d[20].isnan().all() and d[torch.arange(70) != 20].isfinite().all()


def test_picks_out_of_range_and_repeated():
    """An entry outside [0, E) is no pick (a dropped token), a repeated one counts twice."""
    say("balance: odd picks")
    x, topk, mask, d0 = _case(90, 9, 4, seed=5, masked=True, add=True)
    topk[::5, 1] = -1
    topk[::6, 2] = 9
    topk[::4, 0] = topk[::4, 3]
    topk[7, 0] = 2 ** 31 - 1
    _check(x, topk, mask, d0, 0.3, 0.1)


def test_in_place_guard_rows_and_graph():
    say("balance in place, in a graph")
    T, E, k = 1200, 64, 6
    x, topk, mask, d0 = _case(T, E, k, seed=6, masked=True, add=True)
    X, K, M = x.cuda(), topk.cuda(), mask.cuda()
    buf = torch.cat([d0, torch.full((5, E), 3.0)]).cuda()
    loss, saved = moe.moe_balance_fwd(X, K, M, 0.1, 0.01)
    want = moe.moe_balance_bwd(X, saved, M, dlogits=d0.cuda())
    got = moe.moe_balance_bwd(X, saved, M, dlogits=buf[:T], out=buf[:T])
    torch.cuda.synchronize()
    assert torch.equal(got, want) and got.data_ptr() == buf.data_ptr() and (buf[T:] == 3).all()

    def step():
        loss, s = moe.moe_balance_fwd(X, K, M, 0.1, 0.01)
        return [loss, s["counts"], s["tokens"], s["mean_prob"], moe.moe_balance_bwd(X, s, M)]

    graph_check(step, lambda: moe.moe_balance_fwd(d0.cuda(), K))


def test_binding_refusals():
    say("balance binding refusals")
    x, k = torch.zeros(4, 8, device="cuda"), torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    loss, s = moe.moe_balance_fwd(x, k)
    for call in (lambda: moe.moe_balance_fwd(x.bfloat16(), k), lambda: moe.moe_balance_fwd(x, k.long()),
                 lambda: moe.moe_balance_fwd(x, k[:2]), lambda: moe.moe_balance_fwd(x, k[0]),
                 lambda: moe.moe_balance_fwd(x, k, torch.ones(4, device="cuda")),
                 lambda: moe.moe_balance_fwd(x, k, torch.ones(3, dtype=torch.bool, device="cuda")),
                 lambda: moe.moe_balance_fwd(x, torch.zeros(4, 9, dtype=torch.int32, device="cuda")),
                 lambda: moe.moe_balance_fwd(x, k, None, float("inf")),
                 lambda: moe.moe_balance_fwd(torch.zeros(4, 65, device="cuda"), k),
                 lambda: moe.moe_balance_bwd(x[:, :4].contiguous(), s), lambda: moe.moe_balance_bwd(x, s, dloss=1.0),
                 lambda: moe.moe_balance_bwd(x, s, dloss=torch.ones(2, device="cuda")),
                 lambda: moe.moe_balance_bwd(x, s, dlogits=x[:2]), lambda: moe.moe_balance_bwd(x, s, out=x.half())):
        with pytest.raises(moe.MoEError):
            call()
