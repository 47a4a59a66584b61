"""RMS norm, balance loss and 128-block 8-bit products, CPU oracle.

TEST INFRASTRUCTURE ONLY (see the package docstring).

The pages give none of the three (parity unpinned); they are read as what is
usual beside the path they describe:

RMS norm      h = x + residual (rounded to the stream's type),
              rstd = (sum_h h^2 / H + eps)^-1/2, y = h rstd gamma;
              g = dy gamma, dx = rstd (g - xh mean_h(g xh)) + dres with
              xh = h rstd, dgamma = sum_t dy xh
balance loss  p = softmax(logits), n tokens that count, f_e = c_e / (n k),
              P_e = sum_t p_te / n, loss = a E sum_e f_e P_e + z sum_t lse_t^2 / n
8 bits        a block of 128 values of a row (of 128 x 128 of a weight) has the
              fp32 scale s = max(amax, 448 2^-126) / 448 and E4M3 codes, the
              nearest to the fp32 quotient v / s (ties to even)

Norm, loss and products are float64 without roundings; the quantizers follow
the two fp32 quotients, so their results are to be met bit for bit.
"""
from __future__ import annotations

import numpy as np
import torch

from .mx import e4m3_decode, e4m3_encode_magnitude

BLOCK = 128
LEAST = np.float32(448.0) * np.float32(2.0 ** -126)


def _d(t):
    return t if t is None else torch.as_tensor(t).double()


def rmsnorm_fwd(h, gamma=None, eps=1e-6) -> dict:
    h, gamma = _d(h), _d(gamma)
    rstd = 1.0 / torch.sqrt((h * h).mean(1) + eps)
    xh = h * rstd[:, None]
    return {"rstd": rstd, "xh": xh, "y": xh if gamma is None else xh * gamma}


def rmsnorm_bwd(dy, h, rstd, gamma=None, dres=None) -> dict:
    dy, h, rstd, gamma, dres = _d(dy), _d(h), _d(rstd), _d(gamma), _d(dres)
    xh = h * rstd[:, None]
    g = dy if gamma is None else dy * gamma
    c = (g * xh).mean(1, keepdim=True)
    dx = rstd[:, None] * (g - xh * c)
    return {"dx": dx if dres is None else dx + dres, "dgamma": (dy * xh).sum(0), "g": g, "xh": xh, "c": c}


def balance(logits, topk, mask=None, coef=0.01, zcoef=0.0, dloss=1.0) -> dict:
    """Loss, counts and gradient, token by token."""
    x = torch.as_tensor(logits).double()
    T, E = x.shape
    k = topk.shape[1]
    live = [t for t in range(T) if mask is None or bool(mask[t])]
    n = max(1, len(live))
    counts = [0] * E
    p = torch.zeros_like(x)
    lse = torch.zeros(T, dtype=torch.float64)
    for t in live:
        for e in topk[t].tolist():
            if 0 <= e < E:
                counts[e] += 1
        top = x[t].max()
        if top == -float("inf"):
            continue
        ex = torch.exp(x[t] - top)
        p[t] = ex / ex.sum()
        lse[t] = top + torch.log(ex.sum())
    f = torch.tensor(counts, dtype=torch.float64) / (n * k)
    P = p.sum(0) / n
    b, z = coef * E * (f * P).sum(), zcoef * (lse * lse).sum() / n
    d = coef * E / n * p * (f - (p * f).sum(1, keepdim=True)) + 2 * zcoef / n * lse[:, None] * p
    return {"loss": b + z, "balance": b, "z": z, "counts": torch.tensor(counts, dtype=torch.int32),
            "tokens": len(live), "mean_prob": P, "dlogits": dloss * d, "p": p, "lse": lse, "f": f}


def _f32(x) -> np.ndarray:
    return torch.as_tensor(x).float().numpy()


def _encode(v: np.ndarray, s: np.ndarray) -> np.ndarray:
    q = (v / s).astype(np.float32)                      # one fp32 division
    mag = np.minimum(np.abs(q.astype(np.float64)), 448.0)
    bad = np.isnan(mag)
    code = e4m3_encode_magnitude(np.where(bad, 0.0, mag)).astype(np.uint8)
    return np.where(bad, np.uint8(0x7F), code | np.where(np.signbit(v), np.uint8(0x80), np.uint8(0)))


def _scale(amax: np.ndarray) -> np.ndarray:
    return np.maximum(amax, LEAST) / np.float32(448.0)


def quantize_rows(x):
    """x [R, C] -> codes uint8 [R, C], scales fp32 [ceil(C/128), R]."""
    v = _f32(x)
    codes, scales = np.empty(v.shape, np.uint8), []
    for c in range(0, v.shape[1], BLOCK):
        b = v[:, c:c + BLOCK]
        s = _scale(np.abs(b).max(1))
        codes[:, c:c + BLOCK] = _encode(b, s[:, None])
        scales.append(s)
    return codes, np.stack(scales)


def quantize_weight(w):
    """w [N, K] -> codes uint8 [N, K], scales fp32 [ceil(N/128), ceil(K/128)]."""
    v = _f32(w)
    N, K = v.shape
    codes = np.empty(v.shape, np.uint8)
    scales = np.empty(((N + 127) // 128, (K + 127) // 128), np.float32)
    for i in range(scales.shape[0]):
        for j in range(scales.shape[1]):
            at = (slice(i * BLOCK, (i + 1) * BLOCK), slice(j * BLOCK, (j + 1) * BLOCK))
            scales[i, j] = _scale(np.abs(v[at]).max())
            codes[at] = _encode(v[at], scales[i, j])
    return codes, scales


def rows_value(codes, scales) -> torch.Tensor:
    C = codes.shape[1]
    s = np.asarray(scales, np.float64).T.repeat(BLOCK, 1)[:, :C]
    return torch.from_numpy(e4m3_decode(codes) * s)


def weight_value(codes, scales) -> torch.Tensor:
    N, K = codes.shape
    s = np.asarray(scales, np.float64).repeat(BLOCK, 0)[:N].repeat(BLOCK, 1)[:, :K]
    return torch.from_numpy(e4m3_decode(codes) * s)


def linear_fwd(x, w, split) -> torch.Tensor:
    """y of the rows that the experts have; x, w values in float64."""
    out, at = [], 0
    for e, n in enumerate(split):
        out.append(x[at:at + n] @ w[e].T)
        at += n
    return torch.cat(out)


def linear_bwd(dy, dyq, x, w, split):
    """(dx from the quantized dy, [dW from dy itself])."""
    dx, dw, at = [], [], 0
    for e, n in enumerate(split):
        dx.append(dyq[at:at + n] @ w[e])
        dw.append(dy[at:at + n].double().T @ x[at:at + n])
        at += n
    return torch.cat(dx), dw
