"""GPU: ScaledSwiGLU by itself against float64, element by element.

Bounds, u = 2^-24: the exponential's argument rounds (|g| u) and the hardware
exponential and reciprocal are off by a few u, so sigmoid is off by at most
(2 |g| + 12) u of itself, products by u each; bf16 outputs add 2^-8.  The
reciprocal of 1 + exp(-g) above 2^126 is below fp32's normal numbers and
counts as 0: sigmoid is then off by at most 2^-126 (FLUSH), and what it is
multiplied with scales that."""
import numpy as np
import pytest
import torch

import mxfp8_block_scaled_top_amd as moe
from oracle import mx as omx
from oracle import sublayer as S
from tests.helpers import need_gpu, np_, say
from tests.test_gpu_layernorm import _graph_check

pytestmark = pytest.mark.gpu

U, TINY, FLUSH, BF = 2.0 ** -24, 1e-37, 2.0 ** -126, torch.bfloat16


@pytest.fixture(autouse=True)
def _gpu():
    need_gpu()


def _randn(*shape, seed, scale=1.0):
    return (torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * scale).to(BF)


def _within(got, ref, bound, what):
    d = (got.double().cpu() - ref).abs()
    bad = ~(d <= bound)
    assert not bad.any(), (what, int(bad.sum()), float((d / bound)[bad].max()))


SIZES = [(1, 8), (2, 14336), (7, 40), (33, 64), (1001, 1408), (130, 2048), (65, 2080), (4, 4096), (300, 96),
         (3, 65536)]


def _fwd(rows, I, with_prob, ckpt, a1):
    prob = torch.rand(rows, generator=torch.Generator().manual_seed(rows)) if with_prob else None
    a2, saved = moe.moe_swiglu_fwd(a1.cuda(), None if prob is None else prob.cuda(), checkpoint=ckpt)
    torch.cuda.synchronize()
    ref = S.swiglu_fwd(a1, prob)
    g = a1[:, :I].double().abs()
    flush = FLUSH * g * a1[:, I:].double().abs()                    # prob <= 1
    _within(a2, ref, ref.abs() * ((2 * g + 16) * U + 2.0 ** -8 * 1.001) + flush + TINY, "a2")
    if ckpt:      # the very bytes of the quantizer
        codes, scales = omx.quantize_rows(a1)
        assert np.array_equal(np_(saved["a1_codes"]), codes) and np.array_equal(np_(saved["a1_scales"]), scales)


def _bwd(rows, I, with_prob, ckpt, a1, da2):
    prob = torch.rand(rows, generator=torch.Generator().manual_seed(rows)) if with_prob else None
    saved = {"a1": a1.cuda()}
    v = a1.double()
    if ckpt:
        codes, scales = omx.quantize_rows(a1)
        saved = {"a1_codes": torch.from_numpy(codes).cuda(), "a1_scales": torch.from_numpy(scales).cuda()}
        v = torch.from_numpy(omx.dequantize_rows(codes, scales)).double()
    da1, dprob = moe.moe_swiglu_bwd(da2.cuda(), saved, None if prob is None else prob.cuda())
    torch.cuda.synchronize()
    ref, dp = S.swiglu_bwd(da2, v, prob)
    g, u = v[:, :I], v[:, I:]
    sig = torch.sigmoid(g)
    p = 1.0 if prob is None else prob.double()[:, None]
    rel = (4 * g.abs() + 30) * U
    sr = sig * rel + FLUSH
    e = torch.cat([(da2.double() * p * u).abs() * (1 + g.abs()) * sr, (da2.double() * p * g).abs() * sr], 1)
    _within(da1, ref, e + 2.0 ** -8 * (ref.abs() + e) + TINY, "da1")
    if prob is None:
        assert dprob is None
    else:      # a chain of at most I/64/8 pieces of 8, 6 steps and 4 waves
        mag = (da2.double() * g * u).abs()
        _within(dprob, dp, (mag * (sr + sig * (I / 64 + 8 + 10) * U)).sum(1) + TINY, "dprob")


@pytest.mark.parametrize("rows,I", SIZES)
@pytest.mark.parametrize("with_prob", [True, False], ids=["prob", "no_prob"])
def test_forward(rows, I, with_prob):
    say(f"swiglu fwd rows={rows} I={I} prob={with_prob}")
    _fwd(rows, I, with_prob, I % 32 == 0, _randn(rows, 2 * I, seed=I, scale=3.0))


@pytest.mark.parametrize("rows,I", SIZES)
@pytest.mark.parametrize("with_prob,ckpt", [(True, False), (True, True), (False, True)],
                         ids=["bf16", "ckpt", "ckpt_no_prob"])
def test_backward(rows, I, with_prob, ckpt):
    if ckpt and I % 32:
        pytest.skip("a checkpoint has whole blocks of 32")
    say(f"swiglu bwd rows={rows} I={I} prob={with_prob} ckpt={ckpt}")
    _bwd(rows, I, with_prob, ckpt, _randn(rows, 2 * I, seed=I, scale=3.0), _randn(rows, I, seed=I + 1))


def test_far_gates_and_zero_blocks():
    """Gates where the exponential over- and underflows, and blocks of zeros."""
    say("swiglu far gates")
    a1 = _randn(8, 256, seed=1, scale=60.0)
    a1[2] = 0
    a1[3, :128] = -200.0
    a1[4, :128] = 200.0
    a1[5, 32:64] = -0.0
    da2 = _randn(8, 128, seed=2)
    _fwd(8, 128, True, True, a1)
    for ckpt in (False, True):
        _bwd(8, 128, True, ckpt, a1, da2)


def test_no_rows():
    say("swiglu rows=0")
    e = torch.empty((0, 128), dtype=BF, device="cuda")
    a2, saved = moe.moe_swiglu_fwd(e, torch.empty(0, device="cuda"), checkpoint=True)
    da1, dprob = moe.moe_swiglu_bwd(a2, saved, torch.empty(0, device="cuda"))
    torch.cuda.synchronize()
    assert a2.shape == (0, 64) and da1.shape == (0, 128) and dprob.shape == (0,)


@pytest.mark.parametrize("I", [96, 4096])
def test_writes_nothing_past_its_rows(I):
    say(f"swiglu guard rows I={I}")
    rows, G = 9, 5
    a1, da2, prob = _randn(rows, 2 * I, seed=3).cuda(), _randn(rows, I, seed=4).cuda(), torch.rand(rows).cuda()
    L, p = moe.lib(), (lambda t: t.data_ptr())
    a2 = torch.full((rows + G, I), 3.0, dtype=BF, device="cuda")
    codes = torch.full((rows + G, 2 * I), 77, dtype=torch.uint8, device="cuda")
    scales = torch.full((rows + G, 2 * I // 32), 78, dtype=torch.uint8, device="cuda")
    da1 = torch.full((rows + G, 2 * I), 9.0, dtype=BF, device="cuda")
    dprob = torch.full((rows + G,), 11.0, device="cuda")
    s = torch.cuda.current_stream().cuda_stream
    assert L.moe_swiglu_fwd(rows, I, p(a1), p(prob), p(a2), p(codes), p(scales), s) == 0
    assert L.moe_swiglu_bwd(rows, I, p(da2), None, p(codes), p(scales), p(prob), p(da1), p(dprob), s) == 0
    torch.cuda.synchronize()
    assert (a2[rows:] == 3).all() and (codes[rows:] == 77).all() and (scales[rows:] == 78).all()
    assert (da1[rows:] == 9).all() and (dprob[rows:] == 11).all()


def test_offsets_past_32_bits():
    say("swiglu with 2^31 elements")
    rows, I, n = 80_000, 14336, 500
    tail, d = _randn(n, 2 * I, seed=5).cuda(), _randn(n, I, seed=6).cuda()
    a1 = torch.ones((rows, 2 * I), dtype=BF, device="cuda")
    a1[-n:] = tail
    prob = torch.ones(rows, device="cuda")
    a2, saved = moe.moe_swiglu_fwd(a1, prob, checkpoint=True)
    b2, s1 = moe.moe_swiglu_fwd(tail, prob[:n], checkpoint=True)
    torch.cuda.synchronize()
    assert torch.equal(a2[-n:], b2)
    for k in s1:
        assert torch.equal(saved[k][-n:], s1[k]), k
    a2[-n:] = d
    da1, dp = moe.moe_swiglu_bwd(a2, saved, prob)
    db1, dq = moe.moe_swiglu_bwd(d, s1, prob[:n])
    torch.cuda.synchronize()
    assert torch.equal(da1[-n:], db1) and torch.equal(dp[-n:], dq)


def test_many_short_rows():
    """More pieces than one launch's slab holds."""
    say("swiglu many rows")
    rows, I = (1 << 22) + 77, 8
    a1 = _randn(4096, 2 * I, seed=7).cuda().repeat(rows // 4096 + 1, 1)[:rows].contiguous()
    a2, saved = moe.moe_swiglu_fwd(a1)
    one, _ = moe.moe_swiglu_fwd(a1[:4096].contiguous())
    prob = torch.ones(rows, device="cuda")
    da1, dp = moe.moe_swiglu_bwd(a2, saved, prob)
    db1, dq = moe.moe_swiglu_bwd(one, {"a1": a1[:4096].contiguous()}, prob[:4096])
    torch.cuda.synchronize()
    k = rows // 4096 * 4096
    assert torch.equal(a2[:k].view(-1, 4096, I), one.expand(k // 4096, -1, -1)) and torch.equal(a2[k:], one[:rows - k])
    assert torch.equal(da1[:k].view(-1, 4096, 2 * I), db1.expand(k // 4096, -1, -1))
    assert torch.equal(dp[k:], dq[:rows - k]) and torch.equal(da1[k:], db1[:rows - k])


def test_in_a_graph_and_same_bits():
    say("swiglu in a graph")
    a1, da2, prob = _randn(333, 2816, seed=8).cuda(), _randn(333, 1408, seed=9).cuda(), torch.rand(333).cuda()

    def step():
        a2, saved = moe.moe_swiglu_fwd(a1, prob, checkpoint=True)
        return [a2, saved["a1_codes"], *moe.moe_swiglu_bwd(da2, saved, prob)]

    _graph_check(step, None, lambda: moe.moe_swiglu_bwd(a1, {"a1": torch.cat([a1, a1], 1)}, prob))


def test_binding_refusals():
    say("swiglu binding refusals")
    a1 = torch.zeros((4, 64), dtype=BF, device="cuda")
    a2, saved = moe.moe_swiglu_fwd(a1, checkpoint=True)
    for call in (lambda: moe.moe_swiglu_fwd(a1.float()), lambda: moe.moe_swiglu_fwd(a1[:, :15].contiguous()),
                 lambda: moe.moe_swiglu_fwd(a1[:, ::2]), lambda: moe.moe_swiglu_fwd(a1, torch.ones(3, device="cuda")),
                 lambda: moe.moe_swiglu_fwd(a1[:, :48].contiguous(), checkpoint=True),
                 lambda: moe.moe_swiglu_bwd(a2, {}), lambda: moe.moe_swiglu_bwd(a2, {"a1": a2}),
                 lambda: moe.moe_swiglu_bwd(a2, {"a1_codes": saved["a1_codes"]}),
                 lambda: moe.moe_swiglu_bwd(a2, saved, torch.ones(4, dtype=torch.float64, device="cuda"))):
        with pytest.raises(moe.MoEError):
            call()
