"""Formula pins of the layer norm and ScaledSwiGLU oracle: against autograd
and against central differences, in float64 on the CPU."""
import pytest
import torch

from oracle import sublayer as S


def _x(*shape, seed=0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed), dtype=torch.float64)


@pytest.mark.parametrize("T,H", [(1, 8), (3, 40), (7, 96)])
@pytest.mark.parametrize("res", [False, True])
def test_layernorm_gradients_are_autograds(T, H, res):
    x, gamma, beta = _x(T, H, seed=1) * 3 + 1, _x(H, seed=2), _x(H, seed=3)
    dy, dres = _x(T, H, seed=4), (_x(T, H, seed=5) if res else None)
    leaves = [t.clone().requires_grad_() for t in (x, gamma, beta)]
    y = torch.nn.functional.layer_norm(leaves[0], (H,), leaves[1], leaves[2], 1e-5)
    out = (y * dy).sum() + ((leaves[0] * dres).sum() if res else 0.0)
    out.backward()
    f = S.layernorm_fwd(x, gamma, beta, 1e-5)
    b = S.layernorm_bwd(dy, f["xh"], f["rstd"], gamma, dres)
    assert torch.allclose(f["y"], y.detach(), rtol=1e-12, atol=1e-12)
    for got, leaf in zip((b["dx"], b["dgamma"], b["dbeta"]), leaves):
        assert torch.allclose(got, leaf.grad, rtol=1e-10, atol=1e-11)


def test_layernorm_gradient_is_the_difference_quotient():
    T, H, h = 2, 16, 1e-6
    x, gamma, beta, dy = _x(T, H, seed=1), _x(H, seed=2), _x(H, seed=3), _x(T, H, seed=4)
    f = S.layernorm_fwd(x, gamma, beta)
    b = S.layernorm_bwd(dy, f["xh"], f["rstd"], gamma)
    loss = lambda x, g, b: (S.layernorm_fwd(x, g, b)["y"] * dy).sum()      # noqa: E731
    for which, got in ((0, b["dx"]), (1, b["dgamma"]), (2, b["dbeta"])):
        for i in range(got.numel()):
            lo, hi = [x.clone(), gamma.clone(), beta.clone()], [x.clone(), gamma.clone(), beta.clone()]
            lo[which].view(-1)[i] -= h
            hi[which].view(-1)[i] += h
            # error of the quotient: h^2 of the third derivative plus rounding 2^-52 |loss| / h
            assert abs((loss(*hi) - loss(*lo)) / (2 * h) - got.reshape(-1)[i]) < 1e-7


@pytest.mark.parametrize("with_prob", [False, True])
def test_swiglu_gradients(with_prob):
    rows, I = 5, 24
    a1, da2 = _x(rows, 2 * I, seed=1) * 2, _x(rows, I, seed=2)
    prob = torch.rand(rows, generator=torch.Generator().manual_seed(3), dtype=torch.float64) if with_prob else None
    l1 = a1.clone().requires_grad_()
    lp = prob.clone().requires_grad_() if with_prob else torch.ones(rows, dtype=torch.float64, requires_grad=True)
    a2 = torch.nn.functional.silu(l1[:, :I]) * l1[:, I:] * lp[:, None]
    (a2 * da2).sum().backward()
    assert torch.allclose(S.swiglu_fwd(a1, prob), a2.detach(), rtol=1e-12, atol=1e-13)
    da1, dp = S.swiglu_bwd(da2, a1, prob)
    assert torch.allclose(da1, l1.grad, rtol=1e-10, atol=1e-12)
    assert torch.allclose(dp, lp.grad, rtol=1e-10, atol=1e-12)
    h = 1e-6
    for i in (0, 7, 24, 50, 239):
        lo, hi = a1.clone(), a1.clone()
        lo.view(-1)[i] -= h
        hi.view(-1)[i] += h
        q = ((S.swiglu_fwd(hi, prob) - S.swiglu_fwd(lo, prob)) * da2).sum() / (2 * h)
        assert abs(q - da1.reshape(-1)[i]) < 1e-7
