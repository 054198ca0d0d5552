"""The sub-layer of examples/experts_sublayer.py with fewer tokens than it has
buffers for: its workspace is enough for every number of them (a call of fewer
rows can need more), and such a step gives the bits of a layer made for it."""

import os
import sys

import pytest
import torch

from tests.conftest import ROOT

sys.path.insert(0, os.path.join(ROOT, "examples"))

SIZES = dict(hidden=1024, inner=4096, experts=8, top=2, ranks=4)


def test_workspace_is_enough_for_fewer_tokens():
    import experts_sublayer

    import quantized_compression_tensor_amd as T
    f, have = SIZES["inner"] // SIZES["ranks"], experts_sublayer.ExpertsSublayer(300, **SIZES, device="cpu").ws.numel()

    def need(t):
        return max(T.taco_grouped_gated_linear_workspace_bytes(8, 2 * t, f, 1024),
                   T.taco_grouped_linear_workspace_bytes(8, 2 * t, 1024, f),
                   T.taco_grouped_linear_backward_workspace_bytes(8, 2 * t, 1024, f),
                   T.taco_grouped_gated_linear_backward_workspace_bytes(8, 2 * t, f, 1024),
                   T.taco_layer_norm_backward_workspace_bytes(t, 1024))
    assert any(need(t) > need(300) for t in range(1, 300))
    refused = [t for t in range(1, 301) if need(t) > have]
    assert not refused


@pytest.mark.gpu
@pytest.mark.parametrize("tokens", [1, 2, 25, 100, 259])
def test_steps_of_fewer_tokens(tokens):
    import experts_sublayer
    g = torch.Generator(device="cuda")
    g.manual_seed(tokens)
    x = torch.randn(tokens, 1024, generator=g, device="cuda").to(torch.bfloat16)
    dy = torch.randn(tokens, 1024, generator=g, device="cuda").to(torch.bfloat16)
    results = []
    for most in (300, tokens):
        layer = experts_sublayer.ExpertsSublayer(most, **SIZES, shared=1024)
        results.append([layer.forward(x, shared=True), layer.forward(x), layer.backward(x, dy), *layer.dw_in, *layer.dw_out,
                        layer.dgamma, layer.dbeta])
    torch.cuda.synchronize()
    for a, b in zip(*results):
        assert torch.equal(a, b) and bool(torch.isfinite(a).all())
