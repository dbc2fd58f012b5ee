"""The references of the layer operators against the other ones (no GPU)."""
import numpy as np
import pytest
import torch

from tests import layer_util, train_util


@pytest.mark.parametrize("kind", ["normal", "wide", "grid", "tiny", "bad"])
def test_quantize_is_that_of_single_blocks(kind):
    g = torch.Generator().manual_seed(3)
    x = torch.randn(17, 300, generator=g)
    if kind == "wide":
        x = x * torch.exp2(torch.randint(-60, 60, x.shape, generator=g).float())
    if kind == "grid":
        x = torch.randint(-480, 481, x.shape, generator=g).float() / 16.0
    if kind == "tiny":
        x = x * 2.0 ** -130
    if kind == "bad":
        x[2, 5], x[3, 290], x[4] = float("nan"), -float("inf"), 0.0
    x = x.double().numpy()
    for a, b in zip(layer_util.quantize(x), train_util.quantize(x)):
        assert np.array_equal(a, b)


def test_norm_gradient_is_that_of_autograd():
    g = torch.Generator().manual_seed(5)
    h, w = torch.randn(6, 50, generator=g, dtype=torch.float64).requires_grad_(), torch.randn(50, generator=g, dtype=torch.float64).requires_grad_()
    dy, dres = torch.randn(6, 50, generator=g, dtype=torch.float64), torch.randn(6, 50, generator=g, dtype=torch.float64)
    rstd = (h.square().mean(dim=1) + 1e-5).rsqrt()
    ((h * rstd[:, None] * w * dy).sum() + (h * dres).sum()).backward()
    dh, dw, _, _ = layer_util.norm_grad(dy, h.detach(), rstd.detach(), w.detach(), dres)
    assert torch.allclose(dh, h.grad, rtol=1e-12, atol=1e-12) and torch.allclose(dw, w.grad, rtol=1e-12, atol=1e-12)


def test_gate_gradients_are_those_of_autograd():
    g = torch.Generator().manual_seed(6)
    p, q, da = (torch.randn(5, 40, generator=g, dtype=torch.float64) for _ in range(3))
    p.requires_grad_(), q.requires_grad_()
    (torch.nn.functional.silu(p) * q * da).sum().backward()
    dg, du, basis = layer_util.gate_backward(da, p.detach(), q.detach())
    assert torch.allclose(layer_util.gate_forward(p, q), torch.nn.functional.silu(p) * q)
    assert torch.allclose(dg, p.grad, rtol=1e-12, atol=1e-14) and torch.allclose(du, q.grad, rtol=1e-12, atol=1e-14)
    assert bool((dg.abs() <= basis * (1 + 1e-12)).all())
