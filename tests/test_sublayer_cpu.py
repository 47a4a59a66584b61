"""Host-side refusals of the layer norm and the ScaledSwiGLU calls, before any
launch (no GPU needed), at the C entry points and in the binding."""
import ctypes
import os

import pytest
import torch

import mxfp8_block_scaled_top_amd as moe

NULL, SHAPE, ALIGN, WS, ARG = 1, 2, 3, 4, 7
P = ctypes.c_void_p(4096)       # never dereferenced: every call below fails validation
MIS = ctypes.c_void_p(4104)


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(moe.LIB_PATH):
        from mxfp8_block_scaled_top_amd import build
        build.build()
    return moe.lib()


def _ln_fwd(L, **k):
    a = dict(xt=0, wt=1, T=4, H=64, x=P, gamma=P, beta=P, eps=1e-5, y=P, mean=P, rstd=P, codes=P,
             scales=P) | k
    return L.moe_layernorm_fwd(*a.values(), None)


def _ln_bwd(L, **k):
    a = dict(xt=0, wt=1, T=4, H=64, dy=P, x=P, mean=P, rstd=P, codes=None, scales=None, gamma=P,
             dres=P, dx=P, dgamma=P, dbeta=P, ws=P, n=1 << 30) | k
    return L.moe_layernorm_bwd(*a.values(), None)


@pytest.mark.parametrize("change,status", [
    ({"xt": 2}, ARG), ({"wt": -1}, ARG), ({"codes": None}, ARG), ({"scales": None}, ARG),
    ({"eps": -1.0}, ARG), ({"eps": float("nan")}, ARG),
    ({"T": -1}, SHAPE), ({"T": 1 << 31}, SHAPE), ({"H": 0}, SHAPE), ({"H": 12}, SHAPE),
    ({"H": 32768 + 32}, SHAPE), ({"H": 40}, SHAPE),
    ({"x": None}, NULL), ({"y": None}, NULL),
    ({"x": MIS}, ALIGN), ({"gamma": MIS}, ALIGN), ({"beta": MIS}, ALIGN), ({"y": MIS}, ALIGN),
    ({"codes": MIS}, ALIGN),
])
def test_layernorm_fwd_refuses(L, change, status):
    assert _ln_fwd(L, **change) == status


@pytest.mark.parametrize("change,status", [
    ({"xt": 7}, ARG), ({"wt": 2}, ARG), ({"codes": P}, ARG), ({"scales": P}, ARG),
    ({"T": -1}, SHAPE), ({"H": 12}, SHAPE), ({"H": 32776}, SHAPE),
    ({"H": 40, "codes": P, "scales": P}, SHAPE),
    ({"dy": None}, NULL), ({"dx": None}, NULL), ({"rstd": None}, NULL), ({"x": None}, NULL),
    ({"mean": None}, NULL), ({"ws": None}, NULL),
    ({"dy": MIS}, ALIGN), ({"x": MIS}, ALIGN), ({"dres": MIS}, ALIGN), ({"dx": MIS}, ALIGN),
    ({"dgamma": MIS}, ALIGN), ({"dbeta": MIS}, ALIGN), ({"gamma": MIS}, ALIGN), ({"ws": MIS}, ALIGN),
    ({"n": 16}, WS), ({"n": 16, "dgamma": None}, WS),
])
def test_layernorm_bwd_refuses(L, change, status):
    assert _ln_bwd(L, **change) == status


def test_layernorm_workspace_bytes(L):
    f = L.moe_layernorm_workspace_bytes
    assert f(4, 64) >= 2 * 64 * 4 and f(0, 64) > 0
    assert f(-1, 64) == 0 and f(4, 12) == 0 and f(4, 0) == 0 and f(4, 65536) == 0
    # one partial row of 2H floats per workgroup, whatever the batch
    assert f(1 << 30, 4096) == f(1 << 20, 4096)


@pytest.mark.parametrize("change,status", [
    ({"codes": None}, ARG), ({"scales": None}, ARG), ({"rows": -1}, SHAPE), ({"I": 12}, SHAPE),
    ({"I": 40}, SHAPE), ({"I": (1 << 20) + 32}, SHAPE), ({"a1": None}, NULL), ({"a2": None}, NULL),
    ({"a1": MIS}, ALIGN), ({"a2": MIS}, ALIGN), ({"codes": MIS}, ALIGN),
])
def test_swiglu_fwd_refuses(L, change, status):
    a = dict(rows=4, I=64, a1=P, prob=P, a2=P, codes=P, scales=P) | change
    assert L.moe_swiglu_fwd(*a.values(), None) == status


@pytest.mark.parametrize("change,status", [
    ({"codes": P, "scales": P}, ARG), ({"codes": P}, ARG), ({"rows": 1 << 31}, SHAPE),
    ({"I": 4}, SHAPE), ({"a1": None}, NULL), ({"da2": None}, NULL), ({"da1": None}, NULL),
    ({"a1": None, "codes": P, "scales": P, "I": 40}, SHAPE),
    ({"da2": MIS}, ALIGN), ({"a1": MIS}, ALIGN), ({"da1": MIS}, ALIGN),
])
def test_swiglu_bwd_refuses(L, change, status):
    a = dict(rows=4, I=64, da2=P, a1=P, codes=None, scales=None, prob=P, da1=P, dprob=P) | change
    assert L.moe_swiglu_bwd(*a.values(), None) == status


def test_binding_refuses_host_tensors():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    saved = {"mean": torch.zeros(4), "rstd": torch.zeros(4)}
    for call in (lambda: moe.moe_layernorm_fwd(x), lambda: moe.moe_layernorm_bwd(x, saved, x=x),
                 lambda: moe.moe_swiglu_fwd(x), lambda: moe.moe_swiglu_bwd(x, {"a1": x}),
                 lambda: moe.moe_layernorm_fwd(None), lambda: moe.moe_swiglu_fwd(x[0])):
        with pytest.raises(moe.MoEError):
            call()


def _mlp(L, bwd, **k):
    saved = moe._Saved(None, 4096, 4096, 4096, 4096, 4096)
    tab = (ctypes.c_void_p * 2)(4096, 4096)
    common = dict(prec=0, E=2, H=128, I=256, rows=8)
    if bwd:
        a = common | dict(dyp=P, src=None, xp=P, split=P, w1=tab, w2=tab, prob=P, saved=ctypes.byref(saved),
                          codes=P, scales=P, dxp=P, dw1=tab, dw2=tab, dprob=P, ws=P, n=1 << 30) | k
        return L.grouped_mlp_bwd_ckpt(*a.values(), None)
    a = common | dict(xp=P, src=None, split=P, w1=tab, w2=tab, prob=P, yp=P, saved=ctypes.byref(saved),
                      codes=P, scales=P, ws=P, n=1 << 30) | k
    return L.grouped_mlp_fwd_ckpt(*a.values(), None)


@pytest.mark.parametrize("bwd", [False, True], ids=["fwd", "bwd"])
@pytest.mark.parametrize("change,status", [
    ({"codes": None}, NULL), ({"scales": None}, NULL), ({"codes": MIS}, ALIGN), ({"scales": MIS}, ALIGN),
    ({"src": P}, ARG), ({"prec": 3}, ARG), ({"H": 100}, SHAPE), ({"I": 200}, SHAPE), ({"E": 65}, SHAPE),
    ({"rows": -1}, SHAPE), ({"split": None}, NULL), ({"saved": None}, NULL), ({"n": 1}, WS),
])
def test_grouped_mlp_ckpt_refuses(L, bwd, change, status):
    assert _mlp(L, bwd, **change) == status


def test_grouped_mlp_ckpt_needs_no_bf16_a1(L):
    """saved->a1 is NULL above: a call that is refused for its workspace alone got past it."""
    for bwd in (False, True):
        assert _mlp(L, bwd, n=1) == WS
        assert _mlp(L, bwd, prec=1, src=P, n=1) == WS
