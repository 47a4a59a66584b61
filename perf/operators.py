"""Cases, plain forms and calls of the pre-norm and 8-bit-checkpoint operators.

Six operators: layer norm forward and backward (``moe_layernorm_*``), the
scaled SwiGLU on its own (``moe_swiglu_*``) and the grouped expert MLP whose
saved gate_up output is held in 8 bits (``grouped_mlp_*_ckpt``).  A checkpoint
is MXFP8: E4M3 codes with one E8M0 scale per 32 consecutive values of a row,
X = the smallest power of two with amax <= 448 X.

``run`` computes a pass either with elementary torch operations in fp32 (the
plain form) or, with ``own`` set, through the package's entry points.
``exact`` computes the same outputs in fp64 from the definitions.
"""
import math

import numpy as np
import torch

own = False

EPS = 1e-5


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # the norm in front of the router for one generated token
        {"name": "norm_fwd_token", "op": "norm_fwd", "T": 1, "H": 4096, "x": "bf16", "ckpt": False},
        # the norm of a Mixtral-sized training batch, its normalized rows kept in 8 bits
        {"name": "norm_fwd_batch", "op": "norm_fwd", "T": 8192, "H": 4096, "x": "bf16", "ckpt": True},
        # the norm's gradients at the fine-grained layer's batch, from the 8-bit rows
        {"name": "norm_bwd_batch", "op": "norm_bwd", "T": 16384, "H": 2048, "x": "bf16", "ckpt": True, "res": False},
        # an fp32 residual stream of an uneven batch and width, the residual's gradient added in
        {"name": "norm_bwd_uneven_f32", "op": "norm_bwd", "T": 1777, "H": 1416, "x": "f32", "ckpt": False, "res": True},
        # one token's two experts at generation time
        {"name": "swiglu_fwd_token", "op": "swiglu_fwd", "rows": 2, "I": 14336, "ckpt": False, "prob": True},
        # the activation of a Mixtral-sized batch between two grouped linear calls, a1 kept in 8 bits
        {"name": "swiglu_fwd_batch", "op": "swiglu_fwd", "rows": 16384, "I": 14336, "ckpt": True, "prob": True},
        # its backward pass from the 8-bit checkpoint
        {"name": "swiglu_bwd_batch", "op": "swiglu_bwd", "rows": 16384, "I": 14336, "ckpt": True, "prob": True},
        # an uneven small batch of the fine-grained experts, from a bf16 a1
        {"name": "swiglu_bwd_uneven", "op": "swiglu_bwd", "rows": 5003, "I": 1408, "ckpt": False, "prob": True},
        # the Mixtral layer's forward pass in bf16, balanced experts
        {"name": "mlp_fwd_bf16", "op": "mlp_fwd", "precision": "bf16", "rows": 16384, "H": 4096, "I": 14336, "E": 8, "zipf": 0.0},
        # the fine-grained layer's forward pass in MXFP8: 64 experts, Zipf loads, some empty
        {"name": "mlp_fwd_mxfp8_skewed", "op": "mlp_fwd", "precision": "mxfp8", "rows": 32771, "H": 2048, "I": 1408, "E": 64, "zipf": 2.4},
        # the Mixtral layer's backward pass in bf16 on a short uneven batch
        {"name": "mlp_bwd_bf16", "op": "mlp_bwd", "precision": "bf16", "rows": 4099, "H": 4096, "I": 14336, "E": 8, "zipf": 0.5},
        # a handful of rows over fine-grained experts, several of them empty
        {"name": "mlp_bwd_few", "op": "mlp_bwd", "precision": "bf16", "rows": 37, "H": 2048, "I": 1408, "E": 8, "zipf": 2.4},
    ]


def _log(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_bwd", "swiglu_fwd", "swiglu_bwd", "mlp_fwd", "mlp_bwd"])
    ckpt = rng.random() < 0.5
    step = 32 if ckpt else 8
    if op in ("norm_fwd", "norm_bwd"):
        H = _log(rng, 64, 16384, step)
        T = _log(rng, 1, min(65536, (1 << 25) // H))
        c = {"op": op, "T": T, "H": H, "x": rng.choice(["bf16", "f32"]), "ckpt": ckpt}
        if op == "norm_bwd":
            c["res"] = rng.random() < 0.5
        return c
    if op in ("swiglu_fwd", "swiglu_bwd"):
        I = _log(rng, 64, 16384, step)
        rows = _log(rng, 1, min(131072, 16384 * 14336 // I))
        return {"op": op, "rows": rows, "I": I, "ckpt": ckpt, "prob": rng.random() < 0.75}
    H, I = _log(rng, 128, 4096, 128), _log(rng, 128, 8192, 128)
    E = rng.randint(1, 16)
    c = {"op": op, "rows": _log(rng, 1, 8192), "H": H, "I": I, "E": E, "zipf": round(rng.uniform(0.0, 2.4), 2)}
    c["precision"] = rng.choice(["bf16", "mxfp8"]) if op == "mlp_fwd" else "bf16"
    return c


def work(case):
    op = case["op"]
    if op in ("norm_fwd", "norm_bwd"):
        n, xb = case["T"] * case["H"], 2 if case["x"] == "bf16" else 4
        q = 33 / 32
        if op == "norm_fwd":        # x in; y out, and the checkpoint
            b = n * (xb + 2 + (q if case["ckpt"] else 0))
            return {"bytes": b + 8 * case["T"] + 8 * case["H"], "flops": 8 * n}
        # dy and the saved rows in, dx out; the residual's gradient in
        b = n * (2 + (q if case["ckpt"] else xb) + xb + (xb if case["res"] else 0))
        return {"bytes": b + 8 * case["T"] + 16 * case["H"], "flops": 14 * n}
    if op in ("swiglu_fwd", "swiglu_bwd"):
        n, q = case["rows"] * case["I"], 2 * 33 / 32
        if op == "swiglu_fwd":      # a1 in; a2 out, and the checkpoint
            return {"bytes": n * (4 + 2 + (q if case["ckpt"] else 0)), "flops": 8 * n}
        return {"bytes": n * (2 + (q if case["ckpt"] else 4) + 4), "flops": 16 * n}
    rows, H, I = case["rows"], case["H"], case["I"]
    used = min(case["E"], rows)     # an expert without rows needs no weights
    weights = 2 * used * 3 * H * I
    if op == "mlp_fwd":             # xp and weights in; yp and the checkpoint out
        return {"bytes": weights + rows * (4 * H + 2 * I * 33 / 32), "flops": 6 * rows * H * I}
    # dyp, xp, a2, checkpoint and weights in; dxp and every expert's weight gradients out
    return {"bytes": weights + 2 * case["E"] * 3 * H * I + rows * (6 * H + 2 * I + 2 * I * 33 / 32),
            "flops": 12 * rows * H * I}


# ------------------------------------------------------------------ inputs
def _split(case, seed):
    """Rows of each expert: multinomial over Zipf weights in a random order."""
    rng = np.random.default_rng(seed)
    w = np.arange(1, case["E"] + 1, dtype=np.float64) ** -case["zipf"]
    rng.shuffle(w)
    return rng.multinomial(case["rows"], w / w.sum()).astype(np.int32)


def _pow2(s):
    """2^(s - 127) in fp32 from the E8M0 bytes, exactly."""
    return torch.where(s > 0, s.int() << 23, torch.full_like(s, 1 << 22, dtype=torch.int32)).view(torch.float32)


def _mx_codes(t):
    """MXFP8 of fp32 rows: (E4M3 codes, E8M0 scales, the values they stand for)."""
    b = t.reshape(t.shape[0], t.shape[1] // 32, 32)
    m, e = torch.frexp(b.abs().amax(-1))              # amax = m 2^e, m in [1/2, 1)
    s = (e - 9 + (m > 0.875).int() + 127).clamp(0, 254)
    s = torch.where(m == 0, torch.zeros_like(s), s)
    scale = _pow2(s).unsqueeze(-1)
    codes = (b / scale).to(torch.float8_e4m3fn)
    value = (codes.float() * scale).reshape(t.shape)
    return codes.reshape(t.shape), s.to(torch.uint8), value


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    bf, f32 = torch.bfloat16, torch.float32

    def randn(*shape, dtype=bf, std=1.0):
        return torch.randn(*shape, generator=g, device="cuda", dtype=f32).mul_(std).to(dtype)

    op = case["op"]
    s = {"case": dict(case)}
    if op in ("norm_fwd", "norm_bwd"):
        T, H = case["T"], case["H"]
        xt = bf if case["x"] == "bf16" else f32
        # a residual stream: rows of unlike size and mean, a few columns that stand out
        x = randn(T, H, dtype=f32)
        x[:, :: max(1, H // 7)] *= 12.0
        x = x * (0.5 + 3.0 * torch.rand(T, 1, generator=g, device="cuda")) + 0.3 * randn(T, 1, dtype=f32)
        s["x"] = x.to(xt)
        s["gamma"] = 1.0 + randn(H, dtype=f32, std=0.2)
        s["beta"] = randn(H, dtype=f32, std=0.2)
        if op == "norm_bwd":
            xf = s["x"].float()
            mean = xf.mean(1)
            rstd = torch.rsqrt((xf - mean[:, None]).square().mean(1) + EPS)
            s["mean"], s["rstd"] = mean, rstd
            if case["ckpt"]:
                codes, scales, _ = _mx_codes((xf - mean[:, None]) * rstd[:, None])
                s["codes"], s["scales"] = codes.view(torch.uint8), scales
                del s["x"]
            s["dy"] = randn(T, H)
            s["dres"] = randn(T, H, dtype=xt) if case["res"] else None
        return s
    if op in ("swiglu_fwd", "swiglu_bwd"):
        rows, I = case["rows"], case["I"]
        s["a1"] = randn(rows, 2 * I, std=1.5)
        s["prob"] = torch.rand(rows, generator=g, device="cuda") if case["prob"] else None
        if op == "swiglu_bwd":
            s["da2"] = randn(rows, I)
            if case["ckpt"]:
                codes, scales, _ = _mx_codes(s.pop("a1").float())
                s["codes"], s["scales"] = codes.view(torch.uint8), scales
        return s
    rows, H, I, E = case["rows"], case["H"], case["I"], case["E"]
    sizes = _split(case, seed)
    s["sizes"] = sizes.tolist()
    s["split"] = torch.from_numpy(sizes).cuda()
    s["xp"] = randn(rows, H)
    s["w1"] = [randn(2 * I, H, std=H ** -0.5) for _ in range(E)]
    s["w2"] = [randn(H, I, std=I ** -0.5) for _ in range(E)]
    s["prob"] = torch.rand(rows, generator=g, device="cuda")
    if op == "mlp_bwd":
        s["dyp"] = randn(rows, H)
        # what a forward pass leaves: the gate_up output in 8 bits, a2 in bf16
        codes, scales, v = _mx_codes(randn(rows, 2 * I, dtype=f32))
        s["codes"], s["scales"] = codes.view(torch.uint8), scales
        s["a2"] = (s["prob"][:, None] * torch.nn.functional.silu(v[:, :I]) * v[:, I:]).to(bf)
    return s


# ------------------------------------------------------------------ the passes
def _e4m3(codes):
    return codes.view(torch.float8_e4m3fn)


def _e8m0(scales):
    return scales.view(torch.float8_e8m0fnu)


def run(s):
    return (_own if own else _plain)(s)


def _value(codes, scales):
    """The values that MXFP8 rows stand for."""
    v = _e4m3(codes).float().reshape(*scales.shape, 32)
    return (v * _pow2(scales).unsqueeze(-1)).reshape(codes.shape)


def _plain(s):
    c = s["case"]
    return {"norm_fwd": _plain_norm_fwd, "norm_bwd": _plain_norm_bwd, "swiglu_fwd": _plain_swiglu_fwd,
            "swiglu_bwd": _plain_swiglu_bwd, "mlp_fwd": _plain_mlp_fwd, "mlp_bwd": _plain_mlp_bwd}[c["op"]](s, c)


def _plain_norm_fwd(s, c):
    x = s["x"].float()
    mean = x.mean(1)
    d = x - mean[:, None]
    rstd = torch.rsqrt(d.square().mean(1) + EPS)
    xh = d * rstd[:, None]
    out = {"y": (xh * s["gamma"] + s["beta"]).to(torch.bfloat16), "mean": mean, "rstd": rstd}
    if c["ckpt"]:
        codes, scales, _ = _mx_codes(xh)
        out["codes"], out["scales"] = codes, _e8m0(scales)
    return out


def _plain_norm_bwd(s, c):
    dy, rstd = s["dy"].float(), s["rstd"][:, None]
    xh = _value(s["codes"], s["scales"]) if c["ckpt"] else (s["x"].float() - s["mean"][:, None]) * rstd
    g = dy * s["gamma"]
    dx = rstd * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
    if s["dres"] is not None:
        dx = dx + s["dres"].float()
    return {"dx": dx.to(torch.bfloat16 if c["x"] == "bf16" else torch.float32),
            "dgamma": (dy * xh).sum(0), "dbeta": dy.sum(0)}


def _plain_swiglu_fwd(s, c):
    a1, I = s["a1"].float(), c["I"]
    g, u = a1[:, :I], a1[:, I:]
    a2 = g * torch.sigmoid(g) * u
    if s["prob"] is not None:
        a2 = a2 * s["prob"][:, None]
    out = {"a2": a2.to(torch.bfloat16)}
    if c["ckpt"]:
        codes, scales, _ = _mx_codes(a1)
        out["codes"], out["scales"] = codes, _e8m0(scales)
    return out


def _dswiglu(da2, a1, prob, I):
    """(dA1, dprob) in fp32 from dA2 and A1."""
    g, u = a1[:, :I], a1[:, I:]
    sig = torch.sigmoid(g)
    act = g * sig
    d = da2 if prob is None else da2 * prob[:, None]
    da1 = torch.cat([d * u * sig * (1 + g * (1 - sig)), d * act], 1)
    return da1, (da2 * act * u).sum(1)


def _plain_swiglu_bwd(s, c):
    a1 = _value(s["codes"], s["scales"]) if c["ckpt"] else s["a1"].float()
    da1, dprob = _dswiglu(s["da2"].float(), a1, s["prob"], c["I"])
    return {"da1": da1.to(torch.bfloat16), "dprob": None if s["prob"] is None else dprob}


def _plain_mlp_fwd(s, c):
    I, mx = c["I"], c["precision"] == "mxfp8"
    cut = (lambda t: _mx_codes(t)[2]) if mx else (lambda t: t)   # MXFP8 operands, blocks along the contraction
    a1 = torch.cat([cut(x.float()) @ cut(w.float()).T for x, w in zip(s["xp"].split(s["sizes"]), s["w1"])])
    a2 = s["prob"][:, None] * (a1[:, :I] * torch.sigmoid(a1[:, :I]) * a1[:, I:])
    a2 = cut(a2)
    yp = torch.cat([a @ cut(w.float()).T for a, w in zip(a2.split(s["sizes"]), s["w2"])])
    codes, scales, _ = _mx_codes(a1)
    return {"yp": yp.to(torch.bfloat16), "codes": codes, "scales": _e8m0(scales)}


def _plain_mlp_bwd(s, c):
    bf, n = torch.bfloat16, s["sizes"]
    dyp, xp, a2 = s["dyp"].float(), s["xp"].float(), s["a2"].float()
    da2 = torch.cat([d @ w.float() for d, w in zip(dyp.split(n), s["w2"])])
    da1, dprob = _dswiglu(da2, _value(s["codes"], s["scales"]), s["prob"], c["I"])
    dxp = torch.cat([d @ w.float() for d, w in zip(da1.split(n), s["w1"])])
    return {"dxp": dxp.to(bf), "dprob": dprob,
            "dw1": [(d.T @ x).to(bf) for d, x in zip(da1.split(n), xp.split(n))],
            "dw2": [(d.T @ a).to(bf) for d, a in zip(dyp.split(n), a2.split(n))]}


def _own(s):
    import mxfp8_block_scaled_top_amd as moe
    c = s["case"]
    op = c["op"]
    if op == "norm_fwd":
        y, saved = moe.moe_layernorm_fwd(s["x"], s["gamma"], s["beta"], EPS, checkpoint=c["ckpt"])
        out = {"y": y, "mean": saved["mean"], "rstd": saved["rstd"]}
        if c["ckpt"]:
            out["codes"], out["scales"] = _e4m3(saved["xhat_codes"]), _e8m0(saved["xhat_scales"])
        return out
    if op == "norm_bwd":
        saved = {"mean": s["mean"], "rstd": s["rstd"]}
        if c["ckpt"]:
            saved |= {"xhat_codes": s["codes"], "xhat_scales": s["scales"]}
        dx, dgamma, dbeta = moe.moe_layernorm_bwd(
            s["dy"], saved, s["gamma"], x=s.get("x"), dres=s["dres"],
            dx_dtype=torch.bfloat16 if c["x"] == "bf16" else torch.float32)
        return {"dx": dx, "dgamma": dgamma, "dbeta": dbeta}
    if op == "swiglu_fwd":
        a2, saved = moe.moe_swiglu_fwd(s["a1"], s["prob"], checkpoint=c["ckpt"])
        out = {"a2": a2}
        if c["ckpt"]:
            out["codes"], out["scales"] = _e4m3(saved["a1_codes"]), _e8m0(saved["a1_scales"])
        return out
    if op == "swiglu_bwd":
        saved = {"a1_codes": s["codes"], "a1_scales": s["scales"]} if c["ckpt"] else {"a1": s["a1"]}
        da1, dprob = moe.moe_swiglu_bwd(s["da2"], saved, s["prob"])
        return {"da1": da1, "dprob": dprob}
    rows, H, I, E = c["rows"], c["H"], c["I"], c["E"]
    prec = moe.MOE_BF16 if c["precision"] == "bf16" else moe.MOE_MXFP8
    if "ws" not in s:      # buffers that a training program allocates once per shape
        kind = moe.MOE_OP_MLP_FWD if op == "mlp_fwd" else moe.MOE_OP_MLP_BWD
        n = moe.moe_workspace_bytes(kind, rows, H, I, E, 1, prec)
        s["ws"] = torch.empty(max(n, 256), dtype=torch.uint8, device="cuda")
        if op == "mlp_fwd":
            s["saved"] = moe.alloc_saved(rows, H, I, E, prec, "cuda", checkpoint=True)
        else:
            s["saved"] = {"a1_codes": s["codes"], "a1_scales": s["scales"], "a2": s["a2"]}
            s["dw1"] = [torch.empty_like(w) for w in s["w1"]]
            s["dw2"] = [torch.empty_like(w) for w in s["w2"]]
    if op == "mlp_fwd":
        yp, saved = moe.grouped_mlp_fwd_ckpt(s["xp"], s["split"], s["w1"], s["w2"], s["prob"], prec,
                                             s["saved"], s["ws"])
        return {"yp": yp, "codes": _e4m3(saved["a1_codes"]), "scales": _e8m0(saved["a1_scales"])}
    dxp, dw1, dw2, dprob = moe.grouped_mlp_bwd_ckpt(s["dyp"], s["xp"], s["split"], s["w1"], s["w2"], s["prob"],
                                                    s["saved"], prec, s["ws"], s["dw1"], s["dw2"])
    return {"dxp": dxp, "dprob": dprob, "dw1": dw1, "dw2": dw2}


# ------------------------------------------------------------------ 64 bits
def _blocks64(t):
    """MXFP8 rows in fp64 from the definition: (codes' values, scales, values).
    The grid of E4M3 has steps of 2^(e-3) in the binade 2^e, and of 2^-9
    below 2^-6; ties go to the even multiple."""
    b = t.double().reshape(t.shape[0], t.shape[1] // 32, 32)
    top = b.abs().max(-1).values
    # the power of two at or below top / 448, and the next one where it is too small
    k = torch.frexp(top / 448)[1].to(torch.int64) - 1
    k = torch.where(top > 448 * _two64(k), k + 1, k)
    k = torch.where(top > 0, k, torch.full_like(k, -127)).clamp(-127, 127)
    v = b * _two64(-k).unsqueeze(-1)
    binade = (torch.frexp(v)[1].to(torch.int64) - 1).clamp_min(-6)
    binade = torch.where(v == 0, torch.full_like(binade, -6), binade)
    step = _two64(binade - 3)
    q = torch.round(v / step) * step
    return q.reshape(t.shape), _two64(k), (q * _two64(k).unsqueeze(-1)).reshape(t.shape)


def _two64(k):
    """2^k in fp64 for whole k, from its bits."""
    return ((k + 1023) << 52).view(torch.float64)


def _rows64(codes, scales):
    """The fp64 values of E4M3 codes times 2^(scale - 127), from the codes' bits."""
    c = codes.to(torch.int64)
    e, m = (c >> 3) & 15, (c & 7).double()
    mag = torch.where(e == 0, m * 2.0 ** -9, (8 + m) * _two64(e - 10))
    v = torch.where(c >= 128, -mag, mag).reshape(*scales.shape, 32)
    return (v * _two64(scales.to(torch.int64) - 127).unsqueeze(-1)).reshape(codes.shape)


def _swish64(z):
    return z / (1 + torch.exp(-z))


def exact(case, seed):
    s = prepare(case, seed)
    f64 = {k: v.double() for k, v in s.items() if isinstance(v, torch.Tensor) and v.is_floating_point()}
    op = case["op"]
    if op == "norm_fwd":
        x = f64["x"]
        var, mean = torch.var_mean(x, 1, correction=0)
        rstd = (var + EPS) ** -0.5
        xh = (x - mean[:, None]) * rstd[:, None]
        out = {"y": torch.addcmul(f64["beta"], xh, f64["gamma"]), "mean": mean, "rstd": rstd}
        if case["ckpt"]:
            out["codes"], out["scales"], _ = _blocks64(xh)
        return out
    if op == "norm_bwd":
        # dx by the chain rule through mean and variance, dL/dxhat = dy gamma
        if case["ckpt"]:
            xh = _rows64(s["codes"], s["scales"])
        else:
            xh = (f64["x"] - f64["mean"][:, None]) * f64["rstd"][:, None]
        H = case["H"]
        dxh = f64["dy"] * f64["gamma"]
        inner = torch.einsum("th,th->t", dxh, xh) / H
        dx = (dxh - dxh.sum(1)[:, None] / H - xh * inner[:, None]) * f64["rstd"][:, None]
        if s["dres"] is not None:
            dx += f64["dres"]
        return {"dx": dx, "dgamma": torch.einsum("th,th->h", f64["dy"], xh), "dbeta": f64["dy"].sum(0)}
    I = case["I"]
    if op == "swiglu_fwd":
        g, u = f64["a1"].split(I, 1)
        a2 = _swish64(g).mul_(u)
        if s["prob"] is not None:
            a2.mul_(f64["prob"][:, None])
        out = {"a2": a2}
        if case["ckpt"]:
            out["codes"], out["scales"], _ = _blocks64(f64["a1"])
        return out
    if op == "swiglu_bwd":
        a1 = _rows64(s["codes"], s["scales"]) if case["ckpt"] else f64["a1"]
        p = f64["prob"] if s["prob"] is not None else torch.ones(case["rows"], dtype=torch.float64, device="cuda")
        da1, dp = _swiglu_grad64(f64["da2"], a1, p, I)
        return {"da1": da1, "dprob": None if s["prob"] is None else dp}
    at = np.concatenate([[0], np.cumsum(s["sizes"])])
    spans = list(zip(at[:-1].tolist(), at[1:].tolist()))
    if op == "mlp_fwd":
        cut = (lambda t: _blocks64(t)[2]) if case["precision"] == "mxfp8" else (lambda t: t.double())
        yp = torch.empty(case["rows"], case["H"], dtype=torch.float64, device="cuda")
        codes = torch.empty(case["rows"], 2 * I, dtype=torch.float32, device="cuda")     # E4M3 values: exact
        scales = torch.empty(case["rows"], 2 * I // 32, dtype=torch.float64, device="cuda")
        for e, (a, b) in enumerate(spans):
            if a == b:
                continue
            z = torch.mm(cut(s["xp"][a:b]), cut(s["w1"][e]).t())
            q, sc, _ = _blocks64(z)
            codes[a:b], scales[a:b] = q.float(), sc
            h = _swish64(z[:, :I]) * z[:, I:] * f64["prob"][a:b, None]
            yp[a:b] = torch.mm(cut(h), cut(s["w2"][e]).t())
        return {"yp": yp, "codes": codes, "scales": scales}
    dxp = torch.empty(case["rows"], case["H"], dtype=torch.float64, device="cuda")
    dprob = torch.empty(case["rows"], dtype=torch.float64, device="cuda")
    dw1, dw2 = [], []
    for e, (a, b) in enumerate(spans):
        dy, w1, w2 = f64["dyp"][a:b], s["w1"][e].double(), s["w2"][e].double()
        da1, dprob[a:b] = _swiglu_grad64(torch.mm(dy, w2), _rows64(s["codes"][a:b], s["scales"][a:b]),
                                         f64["prob"][a:b], I)
        dxp[a:b] = torch.mm(da1, w1)
        dw1.append(torch.mm(da1.t(), f64["xp"][a:b]))
        dw2.append(torch.mm(dy.t(), f64["a2"][a:b]))
    return {"dxp": dxp, "dprob": dprob, "dw1": dw1, "dw2": dw2}


def _swiglu_grad64(da2, a1, p, I):
    """d(p swish(g) u): swish'(g) = swish(g) + sigma(g) (1 - swish(g))."""
    g, u = a1.split(I, 1)
    sw = _swish64(g)
    sigma = 1 / (1 + torch.exp(-g))
    pd = p[:, None] * da2
    dg = pd * u * (sw + sigma * (1 - sw))
    return torch.cat([dg, pd * sw], 1), torch.einsum("ti,ti,ti->t", da2, sw, u)
