"""Products by group and of codes in arrays of more than 2^32 bytes, and their
workspaces between guard elements."""

import pytest
import torch

import quantized_compression_tensor_amd as T
from tests.layers_util import DEV, Out, generator
from tests.test_experts import CASES, Rows, three, whole, whole3
from tests.test_int8 import codes, powers, quantized
from tests.test_layers_large import Space
from tests.test_layers_linear import BF, F, NONE, RELU

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("c", [c for c in CASES if c.M > 32 and (c.M < 400 or c.pad)], ids=lambda c: c.name)
def test_workspaces_by_group(c):
    """Exactly the stated bytes, for arrays of any alignment: the case's, and aligned ones."""
    gen = generator(c.M + c.N)
    for pad, offset in ((c.pad, c.offset), (-c.K % 8, 0)):
        x, w = whole(gen, c.M, c.K, 2, pad, offset), whole3(gen, c.G, c.N, c.K, 2, pad, offset)
        d = whole(gen, c.M, c.N, 2)
        ws = Space((T.taco_grouped_linear_workspace_bytes(c.G, c.M, c.N, c.K) + 3) // 4 * 4)
        out = Rows(c.M, c.N, F)
        T.taco_grouped_linear(x, w, c.offsets(), out.t, act=RELU, workspace=ws.t)
        torch.cuda.synchronize()
        ws.check()
        out.check_rows(c.inside(), "out")
        ws = Space((T.taco_grouped_linear_backward_workspace_bytes(c.G, c.M, c.N, c.K) + 3) // 4 * 4)
        dx, dw, db = Rows(c.M, c.K, F), Out(c.G * c.N, c.K, F), Out(c.G, c.N, F)
        T.taco_grouped_linear_backward(d, x, w, c.offsets(), act=RELU, preact=d, dx=dx.t, dw=three(dw.t, c.G), dbias=db.t,
                                       workspace=ws.t)
        torch.cuda.synchronize()
        ws.check()
        dx.check_rows(c.inside(), "dx")
        dw.check("dw")
        db.check("dbias")


@pytest.mark.parametrize("M,N,K,pad", [(100, 300, 4112, 0), (100, 300, 4111, 3), (700, 1000, 1000, 0), (200, 4096, 512, 3),
                                       (4100, 4104, 4112, 0), (2000, 2004, 900, 1)])
def test_workspaces_of_codes(M, N, K, pad):
    gen = generator(M + N + K)
    x, w = codes(gen, M, K, 3, pad), codes(gen, N, K, 3, pad)
    xs, ws_ = powers(gen, M), powers(gen, N)
    out, half = Out(M, N, F), Out(M, N // 2, F)
    ws = Space((T.taco_linear_int8_workspace_bytes(M, N, K) + 3) // 4 * 4)
    T.taco_linear_int8(x, xs, w, ws_, out.t, workspace=ws.t)
    torch.cuda.synchronize()
    ws.check()
    out.check("out")
    ws = Space((T.taco_gated_linear_int8_workspace_bytes(M, N // 2, K) + 3) // 4 * 4)
    T.taco_gated_linear_int8(x, xs, w, ws_, half.t, act=NONE, workspace=ws.t)
    torch.cuda.synchronize()
    ws.check()
    half.check("gated")


@pytest.mark.parametrize("rows,pad", [(40, 0), (40, 1), (4, 0), (4, 1), (6000, 0)])
def test_weights_beyond_32_bits(rows, pad):
    """1024 experts' weights and gradients are 2.2e9 elements; the first, one in
    the middle and the last have rows."""
    G, N, K = 1024, 1024, 2096 + pad
    gen = generator(rows)
    w = torch.zeros(G, N, K, dtype=BF, device=DEV)
    used = (0, 511, 1023)
    for g in used:
        w[g] = torch.randint(-2, 3, (N, K), generator=gen, device=DEV)
    cuts = [0, rows // 3, rows // 2, rows]
    o = torch.zeros(G + 1, dtype=torch.int32, device=DEV)
    o[1:], o[512:], o[1024] = cuts[1], cuts[2], cuts[3]
    x, d = whole(gen, rows, K, 2), whole(gen, rows, N, 2)
    out, dx = Out(rows, N, F), Out(rows, K, F)
    dw, db = torch.full_like(w, 7), torch.full((G, N), 7.0, device=DEV)
    T.taco_grouped_linear(x, w, o, out.t, workspace=Space((T.taco_grouped_linear_workspace_bytes(G, rows, N, K) + 3) // 4 * 4).t)
    T.taco_grouped_linear_backward(d, x, w, o, dx=dx.t, dw=dw, dbias=db, workspace=Space(
        (T.taco_grouped_linear_backward_workspace_bytes(G, rows, N, K) + 3) // 4 * 4).t)
    torch.cuda.synchronize()
    out.check("out")
    dx.check("dx")
    for g, a, b in zip(used, cuts, cuts[1:]):
        assert torch.equal(out.t[a:b].double(), x[a:b].double() @ w[g].double().t())
        assert torch.equal(dx.t[a:b].double(), d[a:b].double() @ w[g].double())
        assert torch.equal(dw[g], (d[a:b].double().t() @ x[a:b].double()).to(BF))
        assert torch.equal(db[g].double(), d[a:b].double().sum(0))
    others = torch.ones(G, dtype=torch.bool, device=DEV)
    others[list(used)] = False
    assert not bool(db[others].any())
    for first in range(0, G, 64):
        block = dw[first:first + 64].flatten(1).any(1)
        assert not bool(block[others[first:first + 64]].any())


@pytest.mark.parametrize("M,N,K", [(2200, 40, 96), (40, 2200, 96), (3000, 2200, 64)])
def test_rows_of_codes_beyond_32_bits(M, N, K):
    """Rows that lie 2^21 codes apart."""
    gen = generator(M + N)
    ld = T.TACO_LINEAR_MAX_STRIDE
    wide = torch.empty(max(M, N), ld, dtype=torch.int8, device=DEV)
    x, w = wide[:M, :K], wide[:N, K:2 * K]
    x.copy_(torch.randint(-3, 4, (M, K), generator=gen, device=DEV))
    w.copy_(torch.randint(-3, 4, (N, K), generator=gen, device=DEV))
    xs, ws = powers(gen, M), powers(gen, N)
    out = Out(M, N, F)
    T.taco_linear_int8(x, xs, w, ws, out.t, workspace=Space((T.taco_linear_int8_workspace_bytes(M, N, K) + 3) // 4 * 4).t)
    q, s = wide[:M, 4 * K:5 * K], torch.empty(M, device=DEV)
    T.taco_quantize_rows(out.t[:, :K] if N >= K else out.t.repeat(1, 3)[:, :K].contiguous(), q, s)
    torch.cuda.synchronize()
    out.check("out")
    assert torch.equal(out.t.double(), (x.double() @ w.double().t()) * xs.double()[:, None] * ws.double())
    want_q, want_s = quantized(out.t[:, :K] if N >= K else out.t.repeat(1, 3)[:, :K])
    assert torch.equal(s.cpu(), torch.from_numpy(want_s)) and torch.equal(q.cpu(), torch.from_numpy(want_q))
