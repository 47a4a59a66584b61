"""Layer norm and ScaledSwiGLU by themselves, CPU oracle.

TEST INFRASTRUCTURE ONLY (see the package docstring).

Layer norm (the norm in front of the router; the pages do not give it, it is
the layer norm of a pre-norm transformer block: parity unpinned)

  mean = sum_h x / H,  var = sum_h (x - mean)^2 / H,  rstd = (var + eps)^-1/2
  xh = (x - mean) rstd,  y = xh gamma + beta
  g = dy gamma;  dx = rstd (g - mean_h(g) - xh mean_h(g xh)) + dres
  dgamma = sum_t dy xh;  dbeta = sum_t dy

ScaledSwiGLU [BioNeMo, section "MXFP8与融合MLP": SwiGLU times the routing
probability]: a2 = p silu(g) u with [g, u] = a1, and its gradients as in mlp.py.

An 8-bit checkpoint is the MXFP8 of xh or a1 by rows (mx.quantize_rows); the
backward then takes the values that the codes stand for in place of xh or a1.

Everything is float64, nothing is rounded; the formulas are pinned against
autograd and against central differences by the CPU tests.
"""
from __future__ import annotations

import torch


def _d(t):
    return t if t is None else torch.as_tensor(t).double()


def layernorm_fwd(x, gamma=None, beta=None, eps=1e-5) -> dict:
    x, gamma, beta = _d(x), _d(gamma), _d(beta)
    mean = x.mean(1)
    d = x - mean[:, None]
    rstd = 1.0 / torch.sqrt((d * d).mean(1) + eps)
    xh = d * rstd[:, None]
    y = xh if gamma is None else xh * gamma
    return {"mean": mean, "rstd": rstd, "xh": xh, "y": y if beta is None else y + beta}


def layernorm_bwd(dy, xh, rstd, gamma=None, dres=None) -> dict:
    dy, xh, rstd, gamma, dres = _d(dy), _d(xh), _d(rstd), _d(gamma), _d(dres)
    g = dy if gamma is None else dy * gamma
    c1, c2 = g.mean(1, keepdim=True), (g * xh).mean(1, keepdim=True)
    dx = rstd[:, None] * (g - c1 - xh * c2)
    return {"dx": dx if dres is None else dx + dres, "dgamma": (dy * xh).sum(0), "dbeta": dy.sum(0),
            "c1": c1, "c2": c2, "g": g}


def swiglu_fwd(a1, prob=None) -> torch.Tensor:
    a1, prob = _d(a1), _d(prob)
    I = a1.shape[1] // 2
    a2 = a1[:, :I] * torch.sigmoid(a1[:, :I]) * a1[:, I:]
    return a2 if prob is None else a2 * prob[:, None]


def swiglu_bwd(da2, a1, prob=None):
    """(da1, dprob)."""
    da2, a1, prob = _d(da2), _d(a1), _d(prob)
    I = a1.shape[1] // 2
    g, u = a1[:, :I], a1[:, I:]
    sig = torch.sigmoid(g)
    s = g * sig
    d = da2 if prob is None else da2 * prob[:, None]
    return torch.cat([d * u * sig * (1 + g * (1 - sig)), d * s], 1), (da2 * s * u).sum(1)
