"""The sub-layer of examples/experts_sublayer.py at a small size against the same
step in float64: its output, its gradients and those of its weights within the
roundings of its bf16 tensors, its 8-bit codes and the codec of its all-reduce."""

import os
import sys

import pytest
import torch

from tests.conftest import ROOT

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(ROOT, "examples"))


def gated(n, w, f):
    z = n @ w.t()
    return z[:, :f] * torch.sigmoid(z[:, :f]) * z[:, f:]


def step64(layer, x, dy, shared):
    """y and the gradients by automatic differentiation, with the routing that the layer took."""
    v = {k: t.detach().double().requires_grad_(True) for k, t in dict(
        x=x, gamma=layer.gamma, beta=layer.beta, **{f"in{r}": w for r, w in enumerate(layer.w_in)},
        **{f"out{r}": w for r, w in enumerate(layer.w_out)}).items()}
    mean, var = v["x"].mean(1, keepdim=True), v["x"].var(1, unbiased=False, keepdim=True)
    n = (v["x"] - mean) / torch.sqrt(var + 1e-5) * v["gamma"] + v["beta"]
    o, y = layer.offsets.tolist(), torch.zeros_like(v["x"])
    for r in range(layer.ranks):
        for e in range(layer.experts):
            rows = slice(o[e], o[e + 1])
            token, p = layer.token[rows], layer.weight[rows].double()[:, None]
            y = y.index_add(0, token, p * (gated(n[token], v[f"in{r}"][e], layer.f) @ v[f"out{r}"][e].t()))
        if shared:
            (qi, si), (qo, so) = layer.s_in[r], layer.s_out[r]
            h = gated(n, qi.double() * si.double()[:, None], layer.shared)
            y = y + h @ (qo.double() * so.double()[:, None]).t()
    (y * dy.double()).sum().backward()
    return y.detach(), {k: t.grad for k, t in v.items()}


def off(got, want):
    return float((got.double() - want).norm() / want.norm())


@pytest.mark.parametrize("tokens,hidden,inner,experts,top,ranks", [(200, 512, 528, 6, 2, 2), (1, 256, 256, 8, 3, 4)])
def test_sublayer(tokens, hidden, inner, experts, top, ranks):
    import experts_sublayer
    layer = experts_sublayer.ExpertsSublayer(tokens, hidden, inner, experts, top, ranks, shared=256)
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    x = torch.randn(tokens, hidden, generator=g, device="cuda").to(torch.bfloat16)
    dy = torch.randn(tokens, hidden, generator=g, device="cuda").to(torch.bfloat16)
    # between x and an output lie at most eight bf16 roundings of 1.7e-3 each in the mean; a code of 8 bits, of
    # values whose largest of 64 or more is about three deviations, is off by 3 / 127 / sqrt(12) = 0.7e-2, twice in
    # the all-reduce (its sums lose less), and twice in the shared expert
    bf16, codec = 8 * 1.7e-3, 2 * 0.9e-2
    y = layer.forward(x, shared=True)
    want, _ = step64(layer, x, dy, True)
    assert off(y - x, want) <= bf16 + codec + 2 * 0.9e-2 + 0.01
    y = layer.forward(x)
    dx = layer.backward(x, dy)
    torch.cuda.synchronize()
    want, grad = step64(layer, x, dy, False)
    assert off(y - x, want) <= bf16 + codec + 0.01
    assert off(dx - dy, grad["x"]) <= bf16 + codec + 0.01
    assert off(layer.dgamma, grad["gamma"]) <= bf16 + codec + 0.01
    assert off(layer.dbeta, grad["beta"]) <= bf16 + codec + 0.01
    for r in range(ranks):
        assert off(layer.dw_in[r], grad[f"in{r}"]) <= bf16
        assert off(layer.dw_out[r], grad[f"out{r}"]) <= bf16
