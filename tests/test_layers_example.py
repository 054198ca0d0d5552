"""The feed-forward sub-layer of examples/ffn_sublayer.py at a small size,
against the same step in float64: with the partial sums added exactly, within
the roundings of its bf16 tensors; compressed, within the codec's error."""

import os
import sys

import pytest
import torch

from tests.conftest import ROOT

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(ROOT, "examples"))


def step64(layer, x, dy):
    """y, dx and the weights' gradients by automatic differentiation in float64."""
    f = layer.f
    leaves = dict(x=x, gamma=layer.gamma, beta=layer.beta, w_out=layer.w_out,
                  **{f"w_in{r}": w for r, w in enumerate(layer.w_in)})
    v = {k: t.double().requires_grad_(True) for k, t in leaves.items()}
    mean, var = v["x"].mean(1, keepdim=True), v["x"].var(1, unbiased=False, keepdim=True)
    n = (v["x"] - mean) / torch.sqrt(var + 1e-5) * v["gamma"] + v["beta"]
    y = v["x"]
    for r in range(layer.ranks):
        z = n @ v[f"w_in{r}"].t()
        h = z[:, :f] * torch.sigmoid(z[:, :f]) * z[:, f:]
        y = y + h @ v["w_out"][:, r * f:(r + 1) * f].t()
    (y * dy.double()).sum().backward()
    return y.detach(), {k: t.grad for k, t in v.items()}


def off(got, want):
    return float((got.double() - want).norm() / want.norm())


@pytest.mark.parametrize("tokens,hidden,inner,ranks", [(192, 512, 1088, 2), (1, 256, 512, 4)])
def test_sublayer(tokens, hidden, inner, ranks):
    import ffn_sublayer
    layer = ffn_sublayer.Sublayer(tokens, hidden, inner, ranks)
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    x = torch.randn(tokens, hidden, generator=g, device="cuda").to(torch.bfloat16)
    dy = torch.randn(tokens, hidden, generator=g, device="cuda").to(torch.bfloat16)
    y64, grad = step64(layer, x, dy)
    # a bf16 rounding is off by 2^-8 at most and by 1.7e-3 in the mean; between
    # x and the last output lie at most eight, and the sums do not amplify them
    for compressed, bound in ((False, 8 * 1.7e-3), (True, 0.06)):
        y, dx = layer.forward(x, compressed), layer.backward(x, dy, compressed)
        torch.cuda.synchronize()
        assert off(y - x, y64 - x.double()) <= bound + 0.01
        assert off(dx - dy, grad["x"] - dy.double()) <= bound + 0.01
        assert off(layer.w_out * 0 + layer.dw_out, grad["w_out"]) <= 8 * 1.7e-3
        for r in range(ranks):
            assert off(layer.dw_in[r], grad[f"w_in{r}"]) <= 8 * 1.7e-3
        assert off(layer.dgamma, grad["gamma"]) <= bound + 0.01
        assert off(layer.dbeta, grad["beta"]) <= bound + 0.01
