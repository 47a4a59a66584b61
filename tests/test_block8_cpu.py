"""CPU: the oracle of the RMS norm, the balance loss and the 128-block formats
against autograd, differences and brute force; host-side refusals of their
calls, before any launch, at the C entry points and in the binding."""
import ctypes
import os

import numpy as np
import pytest
import torch

import mxfp8_block_scaled_top_amd as moe
from oracle import block8 as B
from oracle.mx import e4m3_decode

NULL, SHAPE, ALIGN, WS, ARG = 1, 2, 3, 4, 7
P = ctypes.c_void_p(4096)       # never dereferenced: every call below fails validation
P2 = ctypes.c_void_p(8192)
MIS = ctypes.c_void_p(4104)
ODD = ctypes.c_void_p(4098)


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(moe.LIB_PATH):
        from mxfp8_block_scaled_top_amd import build
        build.build()
    return moe.lib()


# ------------------------------------------------------------------ the oracle
def test_rmsnorm_against_autograd_and_differences():
    g = torch.Generator().manual_seed(1)
    h = torch.randn(3, 10, generator=g, dtype=torch.float64, requires_grad=True)
    gamma = torch.randn(10, generator=g, dtype=torch.float64, requires_grad=True)
    dy, dres = torch.randn(3, 10, generator=g).double(), torch.randn(3, 10, generator=g).double()

    def f(a, b):
        return ((a * (a.square().mean(1, keepdim=True) + 1e-3) ** -0.5 * b) * dy).sum() + (a * dres).sum()
    f(h, gamma).backward()
    fw = B.rmsnorm_fwd(h.detach(), gamma.detach(), 1e-3)
    r = B.rmsnorm_bwd(dy, h.detach(), fw["rstd"], gamma.detach(), dres)
    assert torch.allclose(r["dx"], h.grad, atol=1e-12) and torch.allclose(r["dgamma"], gamma.grad, atol=1e-12)
    e = torch.zeros(3, 10, dtype=torch.float64)
    e[1, 4] = 1e-6
    d = (f(h.detach() + e, gamma.detach()) - f(h.detach() - e, gamma.detach())) / 2e-6
    assert abs(d - r["dx"][1, 4]) < 1e-7


def test_balance_against_autograd():
    g = torch.Generator().manual_seed(2)
    T, E, k = 9, 5, 2
    x = torch.randn(T, E, generator=g, dtype=torch.float64, requires_grad=True)
    topk = torch.topk(x.detach(), k, 1).indices.int()
    mask = torch.tensor([1, 1, 0, 1, 1, 1, 0, 1, 1])
    r = B.balance(x.detach(), topk, mask, 0.3, 0.2, 1.7)
    live = mask.bool()
    n = int(mask.sum())
    c = torch.bincount(topk[live].reshape(-1).long(), minlength=E)
    assert torch.equal(c.int(), r["counts"]) and r["tokens"] == n and int(c.sum()) == n * k
    p = torch.softmax(x[live], 1)
    loss = 0.3 * E * (c / (n * k) * p.mean(0)).sum() + 0.2 * torch.logsumexp(x[live], 1).square().mean()
    (1.7 * loss).backward()
    assert torch.allclose(r["loss"], loss.detach()) and torch.allclose(r["dlogits"], x.grad, atol=1e-14)


def test_even_loads_give_the_coefficient():
    """f = P = 1/E: the balance loss is its coefficient, and its gradient 0."""
    E = 4
    topk = torch.arange(8).remainder(E).reshape(8, 1).int()
    r = B.balance(torch.zeros(8, E), topk, None, 0.25)
    assert abs(float(r["balance"]) - 0.25) < 1e-15 and r["dlogits"].abs().max() < 1e-17


def test_quantizer_by_brute_force():
    """Codes are the nearest of all E4M3 values to the fp32 quotient, ties to even codes."""
    rng = np.random.default_rng(3)
    v = (rng.standard_normal((4, 200)) * np.exp2(rng.integers(-130, 100, (4, 1)))).astype(np.float32)
    v[0, :5] = [0.0, -0.0, 1.0, -1.0, 0.5]
    x = torch.from_numpy(v).bfloat16()
    codes, scales = B.quantize_rows(x)
    grid = e4m3_decode(np.arange(127))
    xf = x.float().numpy()
    for r in range(4):
        for b in range(2):
            blk = xf[r, b * 128:(b + 1) * 128]
            amax = np.float32(np.abs(blk).max())
            s = np.float32(max(amax, B.LEAST)) / np.float32(448)
            assert scales[b, r] == s
            for j, val in enumerate(blk):
                q = abs(float(np.float32(val / s)))
                d = np.abs(grid - min(q, 448.0))
                best = np.flatnonzero(d == d.min())
                want = best[0] if len(best) == 1 else best[best % 2 == 0][0]
                assert codes[r, b * 128 + j] & 0x7F == want
                assert bool(codes[r, b * 128 + j] & 0x80) == bool(np.signbit(val))


def test_zero_blocks_and_non_finite_blocks():
    x = torch.zeros(3, 256, dtype=torch.bfloat16)
    x[1, 3], x[2, 200] = float("nan"), float("inf")
    codes, scales = B.quantize_rows(x)
    assert not codes[0].any() and scales[0, 0] == np.float32(2.0 ** -126)
    assert np.isnan(scales[0, 1]) and np.isinf(scales[1, 2])
    v = B.rows_value(codes, scales)
    assert v[1, :128].isnan().all() and v[2, 128:].isnan().all() and not v[0].any() and not v[1, 128:].any()


def test_weight_blocks_are_row_blocks_of_equal_scale():
    w = torch.randn(160, 288, generator=torch.Generator().manual_seed(4)).bfloat16()
    codes, scales = B.quantize_weight(w)
    assert scales.shape == (2, 3)
    err = (B.weight_value(codes, scales) - w.double()).abs()
    step = torch.from_numpy(scales.astype(np.float64)).repeat_interleave(128, 0)[:160].repeat_interleave(128, 1)[:, :288]
    assert (err <= torch.maximum(w.double().abs() * 2.0 ** -4, step * 2.0 ** -10) * (1 + 1e-6)).all()


def test_linear_gradients_against_autograd():
    g = torch.Generator().manual_seed(5)
    split = [2, 0, 3]
    x = torch.randn(5, 6, generator=g, dtype=torch.float64, requires_grad=True)
    w = [torch.randn(4, 6, generator=g, dtype=torch.float64, requires_grad=True) for _ in split]
    dy = torch.randn(5, 4, generator=g).double()
    (B.linear_fwd(x, w, split) * dy).sum().backward()
    dx, dw = B.linear_bwd(dy, dy, x.detach(), [t.detach() for t in w], split)
    assert torch.allclose(dx, x.grad)
    for a, t in zip(dw, w):
        assert torch.allclose(a, t.grad if t.grad is not None else torch.zeros_like(t))


# ------------------------------------------------------------------ refusals at the C entry points
@pytest.mark.parametrize("change,status", [
    ({"xt": 2}, ARG), ({"st": 2}, ARG), ({"wt": -1}, ARG), ({"xt": 1}, ARG), ({"st": 1, "res": None}, ARG),
    ({"codes": None}, ARG), ({"scales": None}, ARG), ({"eps": -1.0}, ARG), ({"eps": float("nan")}, ARG),
    ({"T": -1}, SHAPE), ({"T": 1 << 31}, SHAPE), ({"H": 0}, SHAPE), ({"H": 12}, SHAPE), ({"H": 32776}, SHAPE),
    ({"x": None}, NULL), ({"h": None}, NULL), ({"y": None, "codes": None, "scales": None}, NULL),
    ({"x": MIS}, ALIGN), ({"res": MIS}, ALIGN), ({"gamma": MIS}, ALIGN), ({"h": MIS}, ALIGN), ({"y": MIS}, ALIGN),
    ({"codes": MIS}, ALIGN), ({"scales": MIS}, ALIGN),
])
def test_rmsnorm_fwd_refuses(L, change, status):
    a = dict(xt=0, st=0, wt=1, T=4, H=64, x=P, res=P, gamma=P, eps=1e-6, h=P, y=P, rstd=P, codes=P,
             scales=P) | change
    assert L.moe_rmsnorm_fwd(*a.values(), None) == status


@pytest.mark.parametrize("change,status", [
    ({"st": 7}, ARG), ({"wt": 2}, ARG), ({"T": -1}, SHAPE), ({"H": 12}, SHAPE), ({"H": 32776}, SHAPE),
    ({"dy": None}, NULL), ({"h": None}, NULL), ({"rstd": None}, NULL), ({"dx": None}, NULL), ({"ws": None}, NULL),
    ({"dy": MIS}, ALIGN), ({"h": MIS}, ALIGN), ({"gamma": MIS}, ALIGN), ({"dres": MIS}, ALIGN), ({"dx": MIS}, ALIGN),
    ({"branch": MIS}, ALIGN), ({"dgamma": MIS}, ALIGN), ({"ws": MIS}, ALIGN), ({"n": 16}, WS),
])
def test_rmsnorm_bwd_refuses(L, change, status):
    a = dict(st=0, wt=1, T=4, H=64, dy=P, h=P, rstd=P, gamma=P, dres=P, dx=P, branch=P, dgamma=P, ws=P,
             n=1 << 30) | change
    assert L.moe_rmsnorm_bwd(*a.values(), None) == status


@pytest.mark.parametrize("change,status", [
    ({"T": -1}, SHAPE), ({"T": 1 << 30}, SHAPE), ({"E": 0}, SHAPE), ({"E": 65}, SHAPE), ({"k": 0}, SHAPE),
    ({"k": 9}, SHAPE), ({"coef": float("inf")}, ARG), ({"z": float("nan")}, ARG),
    ({"logits": None}, NULL), ({"topk": None}, NULL), ({"losses": None}, NULL), ({"counts": None}, NULL),
    ({"tokens": None}, NULL), ({"ws": None}, NULL), ({"logits": MIS}, ALIGN), ({"ws": MIS}, ALIGN), ({"n": 16}, WS),
])
def test_balance_fwd_refuses(L, change, status):
    a = dict(logits=P, T=4, E=8, k=2, topk=P, mask=P, coef=0.01, z=0.0, losses=P, counts=P, tokens=P, prob=P,
             ws=P, n=1 << 30) | change
    assert L.moe_balance_fwd(*a.values(), None) == status


@pytest.mark.parametrize("change,status", [
    ({"T": -1}, SHAPE), ({"E": 65}, SHAPE), ({"k": 9}, SHAPE), ({"coef": float("nan")}, ARG),
    ({"logits": None}, NULL), ({"counts": None}, NULL), ({"tokens": None}, NULL), ({"out": None}, NULL),
    ({"logits": MIS}, ALIGN), ({"add": MIS}, ALIGN), ({"out": MIS}, ALIGN),
])
def test_balance_bwd_refuses(L, change, status):
    a = dict(logits=P, T=4, E=8, k=2, mask=P, coef=0.01, z=0.0, counts=P, tokens=P, dloss=P, add=P, out=P) | change
    assert L.moe_balance_bwd(*a.values(), None) == status


@pytest.mark.parametrize("change,status", [
    ({"rows": -1}, SHAPE), ({"rows": 1 << 31}, SHAPE), ({"cols": 4}, SHAPE), ({"cols": 12}, SHAPE),
    ({"x": None}, NULL), ({"codes": None}, NULL), ({"scales": None}, NULL), ({"x": MIS}, ALIGN),
    ({"codes": MIS}, ALIGN), ({"scales": MIS}, ALIGN),
])
def test_block_quantize_refuses(L, change, status):
    a = dict(x=P, rows=4, cols=64, codes=P, scales=P) | change
    assert L.fp8_block_quantize(*a.values(), None) == status


def _tab(*p):
    return (ctypes.c_void_p * len(p))(*[t.value if t is not None else None for t in p])


@pytest.mark.parametrize("change,status", [
    ({"n": 0}, SHAPE), ({"n": 65}, SHAPE), ({"N": 4}, SHAPE), ({"K": 12}, SHAPE), ({"N": (1 << 22) + 8}, SHAPE),
    ({"K": (1 << 30) + 8}, SHAPE),
    ({"w": None}, NULL), ({"codes": None}, NULL), ({"scales": None}, NULL), ({"w": _tab(P, None)}, NULL),
    ({"codes_t": _tab(None, P)}, NULL), ({"w": _tab(P, MIS)}, ALIGN), ({"codes": _tab(MIS, P)}, ALIGN),
    ({"codes_t": _tab(MIS, P)}, ALIGN), ({"scales": _tab(P, ODD)}, ALIGN),
])
def test_block_quantize_weights_refuses(L, change, status):
    t = _tab(P, P)
    a = dict(n=2, N=64, K=64, w=t, codes=t, scales=t, codes_t=t) | change
    assert L.fp8_block_quantize_weights(*a.values(), None) == status


BLOCK_SHAPES = [({"E": 0}, SHAPE), ({"E": 65}, SHAPE), ({"N": 0}, SHAPE), ({"N": 48}, SHAPE), ({"K": 16}, SHAPE),
                ({"K": 100}, SHAPE), ({"rows": -1}, SHAPE), ({"rows": 1 << 31}, SHAPE), ({"xr": -1}, SHAPE),
                ({"xr": 9}, SHAPE), ({"N": 1 << 15, "K": 1 << 15}, SHAPE),
                ({"src": P, "xr": 1 << 25, "K": 64}, SHAPE), ({"N": (1 << 22) + 32}, SHAPE), ({"K": 1 << 23}, SHAPE),
                ({"split": None}, NULL)]


@pytest.mark.parametrize("change,status", BLOCK_SHAPES + [
    ({"x": None}, NULL), ({"xs": None}, NULL), ({"wc": None}, NULL), ({"ws": None}, NULL), ({"y": None}, NULL),
    ({"wc": _tab(P, None)}, NULL), ({"ws": _tab(None, P)}, NULL), ({"wc": _tab(P, MIS)}, ALIGN),
    ({"ws": _tab(P, ODD)}, ALIGN), ({"x": MIS}, ALIGN), ({"xs": MIS}, ALIGN), ({"y": MIS}, ALIGN),
])
def test_grouped_linear_block_fwd_refuses(L, change, status):
    t = _tab(P, P)
    a = dict(E=2, N=64, K=96, rows=8, x=P, xs=P, xr=8, src=None, split=P, wc=t, ws=t, y=P) | change
    assert L.grouped_linear_block_fwd(*a.values(), None) == status


@pytest.mark.parametrize("change,status", BLOCK_SHAPES + [
    ({"dy": None}, NULL), ({"x": None}, NULL), ({"xs": None}, NULL), ({"wc": None}, NULL), ({"ws": None}, NULL),
    ({"dw": _tab(P, None)}, NULL), ({"wk": None}, NULL), ({"n": 16}, WS), ({"dy": MIS}, ALIGN),
    ({"dx": MIS}, ALIGN), ({"dw": _tab(P, MIS)}, ALIGN), ({"wc": _tab(MIS, P)}, ALIGN), ({"wk": MIS}, ALIGN),
    ({"dw": _tab(P, P)}, ARG),
])
def test_grouped_linear_block_bwd_refuses(L, change, status):
    t = _tab(P, P)
    a = dict(E=2, N=64, K=96, rows=8, dy=P, x=P, xs=P, xr=8, src=None, split=P, wc=t, ws=t, dx=P, dw=_tab(P, P2),
             wk=P, n=1 << 30) | change
    assert L.grouped_linear_block_bwd(*a.values(), None) == status


@pytest.mark.parametrize("N,K", [(1 << 22, 32), (32, 1 << 22)])
def test_more_tiles_than_an_int_counts_are_refused(L, N, K):
    """(rows / 64 + E) * ceil(widest / 128) up to INT32_MAX: with 32768 blocks and 2 experts 64 * 65533 + 63 rows."""
    t, most = _tab(P, P), 64 * ((2 ** 31 - 1) // 32768 - 2) + 63
    w = moe.moe_workspace_bytes
    assert w(moe.MOE_OP_LINEAR_BLOCK_BWD, most, K, N, 2, 1, 0) > 0
    assert w(moe.MOE_OP_LINEAR_BLOCK_BWD, most + 1, K, N, 2, 1, 0) == 0
    for rows, status in ((most, NULL), (most + 1, SHAPE)):
        assert L.grouped_linear_block_fwd(2, N, K, rows, P, P, rows, None, None, t, t, P, None) == status
        assert L.grouped_linear_block_bwd(2, N, K, rows, P, P, P, rows, None, None, t, t, P, _tab(P, P2), P, 1 << 62,
                                          None) == status


def test_workspace_bytes(L):
    f = L.moe_rmsnorm_workspace_bytes
    assert f(4, 64) >= 64 * 4 and f(0, 64) > 0 and f(-1, 64) == f(4, 12) == f(4, 0) == f(4, 65536) == 0
    assert f(1 << 30, 4096) == f(1 << 20, 4096)
    g = L.moe_balance_workspace_bytes
    assert g(64) > g(1) > 0 and g(0) == g(65) == 0
    w = moe.moe_workspace_bytes
    n = w(moe.MOE_OP_LINEAR_BLOCK_BWD, 100, 96, 64, 4, 1, 0)
    assert n >= 100 * (64 + 4 + 2 * 96)
    assert w(moe.MOE_OP_LINEAR_BLOCK_BWD, 100, 96, 65, 4, 1, 0) == 0
    assert w(moe.MOE_OP_LINEAR_BLOCK_BWD, 100, 96, 64, 4, 2, 0) == 0


def test_binding_refuses_host_tensors():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    f, i = torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32)
    w = {"codes": torch.zeros(2, 32, 64, dtype=torch.uint8), "scales": torch.zeros(2, 1, 1)}
    x8 = {"codes": torch.zeros(4, 64, dtype=torch.uint8), "scales": torch.zeros(1, 4)}
    for call in (lambda: moe.moe_rmsnorm_fwd(x), lambda: moe.moe_rmsnorm_fwd(None),
                 lambda: moe.moe_rmsnorm_bwd(x, {"h": x, "rstd": torch.zeros(4)}),
                 lambda: moe.moe_balance_fwd(f, i), lambda: moe.moe_balance_bwd(f, {}),
                 lambda: moe.fp8_block_quantize(x), lambda: moe.fp8_block_quantize_weights([x]),
                 lambda: moe.fp8_block_quantize_weights([]), lambda: moe.fp8_block_quantize_weights(x[None]),
                 lambda: moe.grouped_linear_block_fwd(x, i, w), lambda: moe.grouped_linear_block_fwd(x8, i, w),
                 lambda: moe.grouped_linear_block_fwd(None, i, w),
                 lambda: moe.grouped_linear_block_bwd(x, x8, i, w)):
        with pytest.raises(moe.MoEError):
            call()
