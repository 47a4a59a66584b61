"""GPU: ScaledSwiGLU with values that are not finite, and between two grouped
linear calls, the way a user builds experts of them."""
import pytest
import torch

import mxfp8_block_scaled_top_amd as moe
from oracle import sublayer as S
from tests.helpers import need_gpu, rel_frob, say

pytestmark = pytest.mark.gpu

BF, INF, NAN = torch.bfloat16, float("inf"), float("nan")


@pytest.fixture(autouse=True)
def _gpu():
    need_gpu()


def _kind(t):
    """0 finite, 1 and 2 the infinities, 3 NaN."""
    t = t.cpu()
    return t.isnan() * 3 + (t == INF) * 1 + (t == -INF) * 2


@pytest.mark.parametrize("g,u", [(INF, 1.0), (INF, -2.0), (-INF, 1.0), (NAN, 1.0), (1.0, INF), (-1.0, INF),
                                 (1.0, NAN), (INF, 0.0), (INF, INF)])
@pytest.mark.parametrize("I", [96, 2080])
def test_non_finite_stays_in_its_element(g, u, I):
    """One (gate, up) pair: a2 and da1 are what the formulas give in float64 there
    and what they were elsewhere; dprob changes in that row alone, the checkpoint
    in that pair's blocks alone."""
    say(f"swiglu with g={g} u={u} I={I}")
    rows, r, c = 9, 4, I - 11
    gen = torch.Generator().manual_seed(I)
    a1, da2 = torch.randn(rows, 2 * I, generator=gen).to(BF).cuda(), torch.randn(rows, I, generator=gen).to(BF).cuda()
    prob = torch.rand(rows, generator=gen).cuda()
    bad = a1.clone()
    bad[r, c], bad[r, I + c] = g, u
    (y0, s0), (y1, s1) = (moe.moe_swiglu_fwd(t, prob, checkpoint=True) for t in (a1, bad))
    (d0, p0), (d1, p1) = (moe.moe_swiglu_bwd(da2, {"a1": t}, prob) for t in (a1, bad))
    torch.cuda.synchronize()
    assert torch.equal(_kind(y1), _kind(S.swiglu_fwd(bad.cpu(), prob.cpu())))
    rd, rp = S.swiglu_bwd(da2.cpu(), bad.cpu(), prob.cpu())
    assert torch.equal(_kind(d1), _kind(rd)) and torch.equal(_kind(p1), _kind(rp))
    there = torch.zeros(rows, I, dtype=torch.bool, device="cuda")
    there[r, c] = True
    assert torch.equal(y1[~there], y0[~there])
    both = torch.cat([there, there], 1)
    assert torch.equal(d1[~both], d0[~both])
    keep = torch.arange(rows, device="cuda") != r
    assert torch.equal(p1[keep], p0[keep])
    block = both.view(rows, -1, 32).any(-1)
    assert torch.equal(s1["a1_scales"][~block], s0["a1_scales"][~block])
    codes = [s["a1_codes"].view(rows, -1, 32)[~block] for s in (s0, s1)]
    assert torch.equal(*codes)


@pytest.mark.parametrize("ckpt", [False, True], ids=["bf16", "ckpt"])
@pytest.mark.parametrize("sizes", [[70, 0, 301, 1], [1, 0, 2]], ids=["many", "few"])
def test_between_grouped_linear_calls(sizes, ckpt):
    """gate_up, ScaledSwiGLU, down and all gradients.  Against autograd in float64
    at most five bf16 roundings of 2^-8 / sqrt(3) in the 2-norm meet in one result
    (a1, a2, da2, da1, its own): 0.005, held to twice that as silu's slope may
    exceed 1.  From the 8-bit a1 the activation's gradient is held to the values
    that the codes stand for."""
    H, I, E, rows = 256, 384, len(sizes), sum(sizes)
    say(f"linear, swiglu, linear sizes={sizes} ckpt={ckpt}")
    g = torch.Generator().manual_seed(rows)
    r = lambda *s, std=1.0: (torch.randn(*s, generator=g) * std).to(BF)     # noqa: E731
    x, dy, prob = r(rows, H), r(rows, H), torch.rand(rows, generator=g)
    w1, w2 = [r(2 * I, H, std=H ** -0.5) for _ in sizes], [r(H, I, std=I ** -0.5) for _ in sizes]
    split = torch.tensor(sizes, dtype=torch.int32).cuda()
    xd, dyd, pd, w1d, w2d = x.cuda(), dy.cuda(), prob.cuda(), [w.cuda() for w in w1], [w.cuda() for w in w2]
    a1 = moe.grouped_linear_fwd(xd, split, w1d)
    a2, saved = moe.moe_swiglu_fwd(a1, pd, checkpoint=ckpt)
    y = moe.grouped_linear_fwd(a2, split, w2d)
    da2, dw2 = moe.grouped_linear_bwd(dyd, a2, split, w2d)
    da1, dprob = moe.moe_swiglu_bwd(da2, saved, pd)
    dx, dw1 = moe.grouped_linear_bwd(da1, xd, split, w1d)
    torch.cuda.synchronize()
    leaves = [t.double().requires_grad_() for t in (x, prob, *w1, *w2)]
    xl, pl, w1l, w2l = leaves[0], leaves[1], leaves[2:2 + E], leaves[2 + E:]
    parts = []
    for xe, pe, a, b in zip(xl.split(sizes), pl.split(sizes), w1l, w2l):
        h = xe @ a.T
        parts.append((pe[:, None] * torch.nn.functional.silu(h[:, :I]) * h[:, I:]) @ b.T)
    out = torch.cat(parts)
    (out * dy.double()).sum().backward()
    errs = {"y": rel_frob(y, out.detach())}
    errs |= {f"dw2 {e}": rel_frob(dw2[e], w2l[e].grad) for e in range(E) if sizes[e]}
    if ckpt:
        v = moe.mxfp8_dequantize(saved["a1_codes"], saved["a1_scales"], rows, 2 * I).cpu()
        rd, rp = S.swiglu_bwd(da2.cpu(), v, prob)
        errs |= {"da1": rel_frob(da1, rd), "dprob": rel_frob(dprob, rp)}
    else:
        errs |= {"dx": rel_frob(dx, xl.grad), "dprob": rel_frob(dprob, pl.grad)}
        errs |= {f"dw1 {e}": rel_frob(dw1[e], w1l[e].grad) for e in range(E) if sizes[e]}
    say("  " + str(errs))
    assert max(errs.values()) <= 1e-2, errs
    for e in range(E):
        if not sizes[e]:
            assert not dw1[e].any() and not dw2[e].any()
