"""GPU: layer_step_block, the run of RMS norm, router, balance loss and 8-bit block experts, stage by stage
against float64 on the stage's own inputs (2-norm, 1e-2: bf16 outputs are off by at most 2^-8 of the largest of
each sum's rounding, the 8-bit operands are the same codes on both sides), and as a whole in a graph."""
import numpy as np
import pytest
import torch

import mxfp8_block_scaled_top_amd as moe
from mxfp8_block_scaled_top_amd.layer import layer_step_block
from oracle import block8 as B
from oracle import route as R
from oracle import sublayer as S
from tests.helpers import need_gpu, np_, rel_frob, say
from tests.test_gpu_rmsnorm import graph_check

pytestmark = pytest.mark.gpu

BF, TOL = torch.bfloat16, 1e-2


@pytest.fixture(autouse=True)
def _gpu():
    need_gpu()


def _setup(T, H, I, E, seed, stream):
    g = torch.Generator().manual_seed(seed)
    rn = lambda *s, sc=1.0: torch.randn(*s, generator=g) * sc        # noqa: E731
    p = {"x": rn(T, H).to(BF), "residual": None if stream is None else (rn(T, H) * 2).to(stream),
         "gamma": 1 + 0.2 * rn(H), "w_router": rn(E, H, sc=H ** -0.5).to(BF)}
    w = {"w1": rn(E, 2 * I, H, sc=H ** -0.5).to(BF), "w2": rn(E, H, I, sc=I ** -0.5).to(BF)}
    h_type = stream or BF
    return p, w, rn(T, H).to(BF), rn(T, H).to(h_type), (torch.rand(T, generator=g) < 0.8)


def _val(q, e):
    return B.weight_value(np_(q["codes"][e]), np_(q["scales"][e]))


@pytest.mark.parametrize("T,H,I,E,k,stream", [(100, 192, 160, 5, 2, torch.float32), (37, 128, 64, 8, 3, BF),
                                              (1, 256, 96, 4, 2, None), (700, 320, 224, 16, 4, torch.float32)])
def test_stage_by_stage(T, H, I, E, k, stream):
    say(f"block layer T={T} H={H} I={I} E={E} k={k} stream={stream}")
    p, w, dy, dres, mask = _setup(T, H, I, E, T, stream)
    w8 = {n: moe.fp8_block_quantize_weights(t.cuda(), transposed=True) for n, t in w.items()}
    args = {n: None if t is None else t.cuda() for n, t in p.items()}
    up = torch.tensor([3.0], device="cuda")
    o = layer_step_block(**args, **w8, k=k, dy=dy.cuda(), dres=dres.cuda(), mask=mask.cuda(), dloss=up)
    torch.cuda.synchronize()
    c = {n: t.cpu() for n, t in o.items() if isinstance(t, torch.Tensor)}
    rt = {n: np_(t) for n, t in o["route"].items()}
    # norm and router
    f = B.rmsnorm_fwd(c["h"], p["gamma"])
    assert rel_frob(c["n"], f["y"]) < TOL
    assert rel_frob(c["logits"], c["n"].double() @ p["w_router"].double().T) < TOL
    ref = R.route(c["logits"].numpy(), k)
    assert np.array_equal(rt["dest_row"], ref["dest_row"]) and np.array_equal(rt["split_sizes"], ref["split_sizes"])
    split, src = rt["split_sizes"].tolist(), torch.from_numpy(rt["src_token"]).long()
    bal = B.balance(c["logits"], torch.from_numpy(rt["topk_expert"]), mask, 0.01, 0.001, 3.0)
    assert rel_frob(c["loss"], bal["loss"]) < 1e-5 and torch.equal(o["balance"]["counts"].cpu(), bal["counts"])
    # experts forward
    n8 = B.rows_value(np_(o["norm_saved"]["codes"]), np_(o["norm_saved"]["scales"]))
    assert rel_frob(n8, f["y"]) < 2.0 ** -4
    w1 = [_val(w8["w1"], e) for e in range(E)]
    w2 = [_val(w8["w2"], e) for e in range(E)]
    assert rel_frob(c["a1"], B.linear_fwd(n8[src], w1, split)) < TOL
    assert rel_frob(c["a2"], S.swiglu_fwd(c["a1"], c["pp"])) < TOL
    a8 = B.rows_value(*B.quantize_rows(c["a2"]))
    assert rel_frob(c["yp"], B.linear_fwd(a8, w2, split)) < TOL
    dest = torch.from_numpy(rt["dest_row"]).long()
    assert rel_frob(c["y"], c["yp"].double()[dest].sum(1)) < TOL
    # backward
    q = lambda t: B.rows_value(*B.quantize_rows(t))                  # noqa: E731
    dyp = dy[src]
    da2, dw2 = B.linear_bwd(dyp, q(dyp), a8, w2, split)
    assert rel_frob(c["dw2"], torch.stack(dw2)) < TOL
    da1, dpp = S.swiglu_bwd(da2.to(BF), c["a1"], c["pp"])
    assert rel_frob(c["dpp"], dpp) < TOL
    da1 = da1.to(BF)
    dxp, dw1 = B.linear_bwd(da1, q(da1), n8[src], w1, split)
    assert rel_frob(c["dw1"], torch.stack(dw1)) < TOL
    dl = torch.from_numpy(R.route_bwd(c["logits"].numpy(), rt["topk_expert"], c["dpp"].numpy()[rt["dest_row"]])).double()
    assert rel_frob(c["dlogits"], dl + bal["dlogits"]) < TOL
    dn = dxp[dest].sum(1) + c["dlogits"].double() @ p["w_router"].double()
    assert rel_frob(c["dn"], dn) < TOL
    assert rel_frob(c["dw_router"], c["dlogits"].double().T @ c["n"].double()) < TOL
    b = B.rmsnorm_bwd(c["dn"], c["h"], f["rstd"], p["gamma"], dres)
    assert rel_frob(c["dx"], b["dx"]) < TOL and rel_frob(c["dgamma"], b["dgamma"]) < TOL
    assert c["dx"].dtype == c["h"].dtype == (stream or BF)
    if stream == torch.float32:
        assert rel_frob(c["dx_branch"], b["dx"]) < TOL and c["dx_branch"].dtype == BF
    else:
        assert o["dx_branch"] is None


def test_forward_alone_and_single_tokens():
    """A batch's tokens one at a time give the batch's rows (the router's picks are theirs alone; the products'
    sums are taken block by block in both, so outputs agree to their last rounding of a1 and yp)."""
    say("block layer, token by token")
    p, w, *_ = _setup(6, 256, 128, 4, 3, torch.float32)
    w8 = {n: moe.fp8_block_quantize_weights(t.cuda()) for n, t in w.items()}
    a = {n: t.cuda() for n, t in p.items()}
    full = layer_step_block(**a, **w8, k=2)
    assert "dx" not in full
    for t in range(6):
        one = layer_step_block(a["x"][t:t + 1], a["residual"][t:t + 1], a["gamma"], a["w_router"], **w8, k=2)
        torch.cuda.synchronize()
        assert torch.equal(one["h"], full["h"][t:t + 1])
        assert rel_frob(one["y"], full["y"][t:t + 1]) < TOL


def test_in_a_graph():
    say("block layer in a graph")
    p, w, dy, dres, mask = _setup(300, 256, 192, 8, 9, torch.float32)
    w8 = {n: moe.fp8_block_quantize_weights(t.cuda(), transposed=True) for n, t in w.items()}
    a = {n: t.cuda() for n, t in p.items()}
    dy, dres, mask = dy.cuda(), dres.cuda(), mask.cuda()

    def step():
        o = layer_step_block(**a, **w8, k=2, dy=dy, dres=dres, mask=mask)
        return [o[n] for n in ("y", "h", "loss", "dx", "dx_branch", "dgamma", "dw1", "dw2", "dw_router", "dlogits")]

    graph_check(step, lambda: layer_step_block(**a, **w8, k=3, dy=dres.to(BF), dres=dres))
