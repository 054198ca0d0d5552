"""One tensor-parallel feed-forward sub-layer with experts, its all-reduces
compressed; the ranks' shards live on one GPU, in turn. Each rank holds an equal
part of every expert's inner columns.

    n = layer_norm(x);  each token goes to its `top` best experts, with weights p
    y = x + sum over ranks of [sum over a token's experts e of
            p_e (act(n Wg_er^T) * (n Wu_er^T)) Wd_er^T  +  shared expert in 8 bits]

Training: the routed experts forward and backward (bf16, products by group).
Serving: with the shared expert, whose weights are 8-bit codes with a scale for
each output channel; its activations are quantised token by token.

    python examples/experts_sublayer.py [--tokens 4096 --hidden 4096 --inner 8192 --experts 16 --top 2 --ranks 8]

prints the time of a training step's directions and of a serving step, for many
tokens and for one."""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import quantized_compression_tensor_amd as T  # noqa: E402

BF16, F32, EPS = torch.bfloat16, torch.float32, 1e-5


class ExpertsSublayer:
    """Weights, and every buffer of a step of up to `tokens` tokens."""

    def __init__(self, tokens, hidden, inner, experts, top, ranks, shared=None, codec=None, seed=0, device="cuda"):
        assert inner % ranks == 0 and (shared is None or shared % ranks == 0)
        self.tokens, self.hidden, self.experts, self.top, self.ranks = tokens, hidden, experts, top, ranks
        self.f, self.shared = inner // ranks, None if shared is None else shared // ranks
        self.codec = codec or T.codec(T.TACO_FMT_INT8_SYM, 64, 0)
        g = torch.Generator(device=device)
        g.manual_seed(seed)

        def normal(*shape, scale):
            return (torch.randn(*shape, generator=g, device=device) * scale).to(BF16)

        def new(*shape, dtype=BF16):
            return torch.empty(*shape, dtype=dtype, device=device)

        def codes(w):
            q, s = new(*w.shape, dtype=torch.int8), new(w.shape[0], dtype=F32)
            T.taco_quantize_rows(w, q, s)
            return q, s

        self.gamma, self.beta = normal(hidden, scale=0.1) + 1, normal(hidden, scale=0.1)
        self.w_router = normal(experts, hidden, scale=hidden ** -0.5)
        # rank r's part of every expert: the gate's rows, then the other projection's; and the projection back
        self.w_in = [normal(experts, 2 * self.f, hidden, scale=hidden ** -0.5) for _ in range(ranks)]
        self.w_out = [normal(experts, hidden, self.f, scale=inner ** -0.5) for _ in range(ranks)]
        rows = tokens * top
        self.n, self.sum = new(tokens, hidden), new(tokens, hidden)
        self.mean, self.rstd = new(tokens, dtype=F32), new(tokens, dtype=F32)
        self.z = [new(rows, 2 * self.f) for _ in range(ranks)]
        self.h = [new(rows, self.f) for _ in range(ranks)]
        self.out, self.dh, self.dx = new(rows, hidden), new(rows, self.f), new(rows, hidden)
        self.partial = [new(tokens, hidden) for _ in range(ranks)]
        self.dw_in, self.dw_out = [torch.empty_like(w) for w in self.w_in], [torch.empty_like(w) for w in self.w_out]
        self.dgamma, self.dbeta = new(hidden, dtype=F32), new(hidden, dtype=F32)
        self.shard = [T.empty_compressed(self.codec, tokens, hidden, device) for _ in range(ranks)]
        self.gathered = T.empty_compressed(self.codec, tokens, hidden, device)
        if self.shared:
            s = self.shared
            self.s_in = [codes(normal(2 * s, hidden, scale=hidden ** -0.5)) for _ in range(ranks)]
            self.s_out = [codes(normal(hidden, s, scale=shared ** -0.5)) for _ in range(ranks)]
            self.nq, self.ns = new(tokens, hidden, dtype=torch.int8), new(tokens, dtype=F32)
            self.sh, self.hq, self.hs = new(tokens, s), new(tokens, s, dtype=torch.int8), new(tokens, dtype=F32)
        # (a step of fewer tokens can need more: where tiles are few, their sums are cut into parts)
        self.ws = new(max(self.workspace_bytes(t) for t in range(1, tokens + 1)), dtype=torch.uint8)

    def workspace_bytes(self, tokens):
        """The most that a call of a step of that many tokens needs."""
        rows, hidden, experts, f, s = tokens * self.top, self.hidden, self.experts, self.f, self.shared
        sizes = [T.taco_grouped_gated_linear_workspace_bytes(experts, rows, f, hidden),
                 T.taco_grouped_linear_workspace_bytes(experts, rows, hidden, f),
                 T.taco_grouped_linear_backward_workspace_bytes(experts, rows, hidden, f),
                 T.taco_grouped_gated_linear_backward_workspace_bytes(experts, rows, f, hidden),
                 T.taco_layer_norm_backward_workspace_bytes(tokens, hidden)]
        if s:
            sizes += [T.taco_gated_linear_int8_workspace_bytes(tokens, s, hidden),
                      T.taco_linear_int8_workspace_bytes(tokens, hidden, s)]
        return max(sizes)

    def route(self, x):
        """The norm, and the tokens' rows sorted by expert: their token, their weight and each expert's first row."""
        t = x.shape[0]
        T.taco_layer_norm(x, self.gamma, self.beta, EPS, self.n[:t], mean=self.mean[:t], rstd=self.rstd[:t])
        best = (self.n[:t].float() @ self.w_router.float().t()).topk(self.top, 1)
        expert, order = best.indices.flatten().sort(stable=True)
        self.token = order // self.top
        self.weight = best.values.softmax(1).flatten()[order]
        self.offsets = torch.searchsorted(expert, torch.arange(self.experts + 1, device=x.device), out_int32=True)
        self.rows = self.n[:t][self.token]

    def all_reduce(self, out, tokens):
        c, cols = self.codec, self.hidden
        for r in range(self.ranks):
            T.taco_compress(c, self.partial[r], tokens, cols, 1.0, self.shard[r])
        T.taco_decompress_reduce(c, self.shard, tokens, cols, c_out=c, requant_out=self.gathered)
        T.taco_decompress(c, self.gathered, tokens, cols, out, out_dtype=1)

    def combine(self, rows, tokens, weight=None):
        """The sum of each token's rows, in float32."""
        v = rows.float() if weight is None else rows.float() * weight[:, None]
        return torch.zeros(tokens, rows.shape[1], device=rows.device).index_add_(0, self.token, v)

    def forward(self, x, shared=False):
        t = x.shape[0]
        n_rows = t * self.top
        self.route(x)
        if shared:
            T.taco_quantize_rows(self.n[:t], self.nq[:t], self.ns[:t])
        for r in range(self.ranks):
            T.taco_grouped_gated_linear(self.rows, self.w_in[r], self.offsets, self.h[r][:n_rows],
                                        preact=None if shared else self.z[r][:n_rows], workspace=self.ws)
            T.taco_grouped_linear(self.h[r][:n_rows], self.w_out[r], self.offsets, self.out[:n_rows], workspace=self.ws)
            routed = self.combine(self.out[:n_rows], t, self.weight)
            if shared:
                T.taco_gated_linear_int8(self.nq[:t], self.ns[:t], *self.s_in[r], self.sh[:t], workspace=self.ws)
                T.taco_quantize_rows(self.sh[:t], self.hq[:t], self.hs[:t])
                T.taco_linear_int8(self.hq[:t], self.hs[:t], *self.s_out[r], self.partial[r][:t], residual=routed,
                                   workspace=self.ws)
            else:
                self.partial[r][:t] = routed
        self.all_reduce(self.sum[:t], t)
        return x + self.sum[:t]

    def backward(self, x, dy):
        """The gradients of x through the experts (the routing is held fixed); those of the weights are left in dw_in,
        dw_out, dgamma and dbeta."""
        t = x.shape[0]
        n_rows = t * self.top
        dout = (dy[self.token].float() * self.weight[:, None]).to(BF16)
        for r in range(self.ranks):
            T.taco_grouped_linear_backward(dout, self.h[r][:n_rows], self.w_out[r], self.offsets, dx=self.dh[:n_rows],
                                           dw=self.dw_out[r], workspace=self.ws)
            T.taco_grouped_gated_linear_backward(self.dh[:n_rows], self.rows, self.w_in[r], self.offsets,
                                                 preact=self.z[r][:n_rows], dx=self.dx[:n_rows], dw=self.dw_in[r],
                                                 workspace=self.ws)
            self.partial[r][:t] = self.combine(self.dx[:n_rows], t)
        self.all_reduce(self.sum[:t], t)
        dx = torch.empty_like(x)
        T.taco_layer_norm_backward(self.sum[:t], x, self.gamma, self.mean[:t], self.rstd[:t], dx=dx, dweight=self.dgamma,
                                   dbias=self.dbeta, workspace=self.ws)
        return dx + dy


def main():
    p = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    for name, value in (("tokens", 4096), ("hidden", 4096), ("inner", 8192), ("experts", 16), ("top", 2), ("ranks", 8),
                        ("steps", 5)):
        p.add_argument("--" + name, type=int, default=value)
    a = p.parse_args()
    layer = ExpertsSublayer(a.tokens, a.hidden, a.inner, a.experts, a.top, a.ranks, shared=a.inner)
    x = torch.randn(a.tokens, a.hidden, device="cuda").to(BF16)
    dy = (torch.randn(a.tokens, a.hidden, device="cuda") * 1e-2).to(BF16)
    one = x[:1].contiguous()
    for name, step in (("forward", lambda: layer.forward(x)), ("backward", lambda: layer.backward(x, dy)),
                       ("serving", lambda: layer.forward(x, shared=True)),
                       ("serving, one token", lambda: layer.forward(one, shared=True))):
        step()
        start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        start.record()
        for _ in range(a.steps):
            step()
        end.record()
        torch.cuda.synchronize()
        print(f"{name}: {start.elapsed_time(end) / a.steps:.3f} ms for {a.ranks} ranks' shards")


if __name__ == "__main__":
    main()
