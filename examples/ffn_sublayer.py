"""One tensor-parallel feed-forward sub-layer, forward and backward, with its
two all-reduces compressed; the ranks' shards live on one GPU, in turn.

    y  = x + sum over ranks of (act(n Wg_r^T) * (n Wu_r^T)) Wd_r^T,   n = layer_norm(x)

Forward: the layer norm, each rank's gated projections and its projection back,
whose bf16 partial sums are compressed, reduced and decoded. Backward: each
rank's gradients; the gradients of n are partial sums again and go the same
way; then the layer norm's.

    python examples/ffn_sublayer.py [--tokens 4096 --hidden 5120 --inner 13824 --ranks 8]

prints the time of each direction and the relative error that the compression
brings (against the same step with the partial sums added in float32)."""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import quantized_compression_tensor_amd as T  # noqa: E402

BF16, F32, EPS = torch.bfloat16, torch.float32, 1e-5


class Sublayer:
    """Weights, and every buffer of the step: nothing is allocated while it runs."""

    def __init__(self, tokens, hidden, inner, ranks, codec=None, seed=0, device="cuda"):
        assert inner % ranks == 0
        self.tokens, self.hidden, self.ranks, self.f = tokens, hidden, ranks, inner // ranks
        self.codec = codec or T.codec(T.TACO_FMT_FP8_DUAL, 128, 1)
        g = torch.Generator(device=device)
        g.manual_seed(seed)

        def normal(*shape, scale):
            return (torch.randn(*shape, generator=g, device=device) * scale).to(BF16)

        def new(*shape, dtype=BF16):
            return torch.empty(*shape, dtype=dtype, device=device)

        self.gamma, self.beta = normal(hidden, scale=0.1) + 1, normal(hidden, scale=0.1)
        # rank r's rows of the gate and the other projection, one after the other
        self.w_in = [normal(2 * self.f, hidden, scale=hidden ** -0.5) for _ in range(ranks)]
        # the projection back, whole: a rank reads its columns in place
        self.w_out = normal(hidden, inner, scale=inner ** -0.5)
        self.n, self.sum = new(tokens, hidden), new(tokens, hidden)
        self.mean, self.rstd = new(tokens, dtype=F32), new(tokens, dtype=F32)
        self.z = [new(tokens, 2 * self.f) for _ in range(ranks)]
        self.h = [new(tokens, self.f) for _ in range(ranks)]
        self.dh = new(tokens, self.f)
        self.partial = [new(tokens, hidden) for _ in range(ranks)]
        self.dw_in = [new(2 * self.f, hidden) for _ in range(ranks)]
        self.dw_out = new(hidden, inner)
        self.dgamma, self.dbeta = new(hidden, dtype=F32), new(hidden, dtype=F32)
        self.shard = [T.empty_compressed(self.codec, tokens, hidden, device) for _ in range(ranks)]
        self.scale_ws = [torch.zeros(T.TACO_WORKSPACE_BYTES, dtype=torch.uint8, device=device) for _ in range(ranks)]
        self.gathered = T.empty_compressed(self.codec, tokens, hidden, device)
        sizes = (T.taco_gated_linear_workspace_bytes(tokens, self.f, hidden),
                 T.taco_linear_workspace_bytes(tokens, hidden, self.f),
                 T.taco_linear_backward_workspace_bytes(tokens, hidden, self.f),
                 T.taco_gated_linear_backward_workspace_bytes(tokens, self.f, hidden),
                 T.taco_layer_norm_backward_workspace_bytes(tokens, hidden))
        self.ws = new(max(sizes), dtype=torch.uint8)

    def columns(self, t, r):
        return t[:, r * self.f:(r + 1) * self.f]

    def all_reduce(self, out, compressed):
        """The sum of the ranks' partial sums, in bf16."""
        if not compressed:
            out.copy_(torch.stack([p.float() for p in self.partial]).sum(0))
            return
        c, rows, cols = self.codec, self.tokens, self.hidden
        for r in range(self.ranks):
            T.taco_compress(c, self.partial[r], rows, cols, T.TACO_SCALE_AUTO, self.shard[r],
                            workspace=self.scale_ws[r])
        T.taco_decompress_reduce(c, self.shard, rows, cols, c_out=c, requant_out=self.gathered)
        T.taco_decompress(c, self.gathered, rows, cols, out, out_dtype=1)

    def forward(self, x, compressed=True):
        T.taco_layer_norm(x, self.gamma, self.beta, EPS, self.n, mean=self.mean, rstd=self.rstd)
        for r in range(self.ranks):
            T.taco_gated_linear(self.n, self.w_in[r], self.h[r], preact=self.z[r], workspace=self.ws)
            T.taco_linear(self.h[r], self.columns(self.w_out, r), self.partial[r], workspace=self.ws)
        self.all_reduce(self.sum, compressed)
        return x + self.sum

    def backward(self, x, dy, compressed=True):
        """The gradients of x; those of the weights are left in dw_in, dw_out, dgamma and dbeta."""
        for r in range(self.ranks):
            T.taco_linear_backward(dy, self.h[r], self.columns(self.w_out, r), dx=self.dh,
                                   dw=self.columns(self.dw_out, r), workspace=self.ws)
            T.taco_gated_linear_backward(self.dh, self.n, self.w_in[r], preact=self.z[r], dx=self.partial[r],
                                         dw=self.dw_in[r], workspace=self.ws)
        self.all_reduce(self.sum, compressed)
        dx = torch.empty_like(x)
        T.taco_layer_norm_backward(self.sum, x, self.gamma, self.mean, self.rstd, dx=dx, dweight=self.dgamma,
                                   dbias=self.dbeta, workspace=self.ws)
        return dx + dy


def main():
    p = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    for name, value in (("tokens", 4096), ("hidden", 5120), ("inner", 13824), ("ranks", 8), ("steps", 5)):
        p.add_argument("--" + name, type=int, default=value)
    a = p.parse_args()
    layer = Sublayer(a.tokens, a.hidden, a.inner, a.ranks)
    x = torch.randn(a.tokens, a.hidden, device="cuda").to(BF16)
    dy = (torch.randn(a.tokens, a.hidden, device="cuda") * 1e-2).to(BF16)

    def off(got, want):
        return float((got.float() - want.float()).norm() / want.float().norm())

    plain_y, plain_dx = layer.forward(x, compressed=False), layer.backward(x, dy, compressed=False)
    y, dx = layer.forward(x), layer.backward(x, dy)
    print(f"compressed against float32 sums: forward {off(y - x, plain_y - x):.2e}, gradient {off(dx - dy, plain_dx - dy):.2e}")
    for name, step in (("forward", lambda: layer.forward(x)), ("backward", lambda: layer.backward(x, dy))):
        step()
        start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        start.record()
        for _ in range(a.steps):
            step()
        end.record()
        torch.cuda.synchronize()
        print(f"{name}: {start.elapsed_time(end) / a.steps:.3f} ms for {a.ranks} ranks' shards of {a.tokens} x {a.hidden}")


if __name__ == "__main__":
    main()
