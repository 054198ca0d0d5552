"""Rows to 8-bit codes, and the projections of codes, against their definitions.

Codes and scales must be the definition's bits. Products of small codes with
scales that are powers of two are exact in float32, so a float32 output must
equal the definition, at every edge of a tile. With real scales a sum of codes,
a whole number, becomes a float with one rounding, each scale is one more and
the bias another: 4 U32 of |z| and U32 of the bias; activations and stores as
in test_layers_linear.py."""

import math

import numpy as np
import pytest
import torch

import quantized_compression_tensor_amd as T
from tests.layers_util import DEV, U32, UNIT, Out, generator, matrix, within
from tests.test_layers_linear import ACTS, BF, F, GELU, NONE, RELU, SILU, SIZES, act64, ids, space, whole

pytestmark = pytest.mark.gpu


def codes(gen, rows, cols, most, pad=0, offset=0):
    """Whole numbers of magnitude up to `most` in an int8 view whose rows lie
    cols + pad bytes apart; what lies between the rows is 85."""
    base = torch.full((offset + rows * (cols + pad) + 32,), 85, dtype=torch.int8, device=DEV)
    v = base[offset:offset + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
    return v.copy_(torch.randint(-most, most + 1, (rows, cols), generator=gen, device=DEV))


def powers(gen, n):
    return torch.exp2(torch.randint(-3, 4, (n,), generator=gen, device=DEV).float())


class Codes:
    """An int8 output of [rows, cols] between guards."""

    def __init__(self, rows, cols, pad=0, offset=0):
        self.lo, self.hi = 4096 + offset, 4096 + offset + rows * (cols + pad)
        self.all = torch.full((self.hi + 4096,), -128, dtype=torch.int8, device=DEV)   # no code of the quantisation
        self.t = self.all[self.lo:self.hi].view(rows, cols + pad)[:, :cols]

    def check(self):
        inside = torch.zeros_like(self.all, dtype=torch.bool)
        rows = self.t.shape[0]
        inside[self.lo:self.hi].view(rows, -1)[:, :self.t.shape[1]] = True
        assert bool((self.all[~inside] == -128).all()), "wrote outside the codes"
        assert not bool((self.all[inside] == -128).any()), "left codes unwritten"


# ----------------------------------------------------------- rows to codes --

def quantized(x):
    """The definition in float32, on the CPU: each step rounded once."""
    v = x.detach().float().cpu().numpy()
    with np.errstate(all="ignore"):
        largest = np.max(np.abs(v), axis=1)               # NaN wins
        finite = np.isfinite(largest)
        zero = finite & (largest < np.float32(2.0 ** -100))
        scale = np.where(zero, np.float32(0), np.where(finite, largest / np.float32(127), largest)).astype(np.float32)
        inv = np.where(finite & ~zero, np.float32(1) / largest * np.float32(127), np.float32(0)).astype(np.float32)
        q = np.rint((np.where(inv[:, None] == 0, np.float32(0), v) * inv[:, None]).astype(np.float32))
    return q.astype(np.int8), scale


def check_quantized(x, pad=0, offset=0):
    rows, cols = x.shape
    q, s = Codes(rows, cols, pad, offset), Out(1, rows, F)
    T.taco_quantize_rows(x, q.t, s.vector())
    torch.cuda.synchronize()
    q.check()
    s.check("scale")
    want_q, want_s = quantized(x)
    assert np.array_equal(s.vector().cpu().numpy(), want_s, equal_nan=True)
    assert np.array_equal(q.t.cpu().numpy(), want_q)


@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])
@pytest.mark.parametrize("rows,cols,pad,offset", [
    (1, 1, 0, 0), (3, 7, 1, 1), (5, 8, 0, 0), (129, 9, 3, 2), (1, 5120, 0, 0), (64, 511, 0, 0), (7, 512, 8, 8),
    (3, 2048, 0, 0), (5, 2049, 3, 1), (6, 4096, 0, 0), (4, 4100, 0, 3), (3, 8192, 0, 0), (3, 8200, 0, 0),
    (2, 16384, 0, 0), (2, 16391, 1, 1), (3, 32768, 0, 0), (2, 32769, 0, 0), (2, 70001, 3, 5), (70000, 24, 0, 0),
    (33, 255, 1, 1), (31, 256, 0, 0), (65, 257, 3, 1), (17, 512, 8, 0), (15, 513, 0, 1), (1000, 205, 0, 0)])
def test_quantize_rows(rows, cols, pad, offset, dtype):
    gen = generator(rows + cols)
    x = matrix(gen, rows, cols, dtype, pad, offset, sigma=3.0)
    x[:: 3] *= torch.exp2(torch.randint(-90, 90, (x[:: 3].shape[0], 1), generator=gen, device=DEV).float()).to(dtype)
    check_quantized(x, pad, offset)


def test_quantize_more_rows_than_workgroups():
    """Rows that a workgroup takes one after the other."""
    x = matrix(generator(5), (1 << 16) * 4 + 13, 3, BF)
    check_quantized(x)
    check_quantized(matrix(generator(6), (1 << 16) + 5, 2056, BF, 8))
    check_quantized(matrix(generator(7), (1 << 16) * 32 + 13, 3, BF))


def test_quantize_rows_of_special_values():
    tiny = 2.0 ** -100
    rows = [[0, 0, 0, -0.0], [tiny, -tiny, tiny / 2, 0], [tiny * 0.99, 0, -tiny * 0.9, 0], [1e-45, -1e-40, 0, 0],
            [math.inf, 1, -1, 0], [-math.inf, math.inf, 0, 2], [math.nan, 5, 1, 0], [1, math.nan, math.inf, -math.inf],
            [3e38, -3.4e38, 1e38, 0], [127, 0.5, 1.5, -2.5], [127, 126.5, -0.5, 63.5], [254, 1, 3, -5], [-7, 7, 0, 1e-30]]
    x = torch.tensor(rows, device=DEV)
    check_quantized(x)
    check_quantized(x.to(BF))
    wide = torch.zeros(len(rows), 40001, device=DEV)     # the last columns of rows that are read twice
    wide[:, -4:] = x
    check_quantized(wide)


# ----------------------------------------------------------------- exactly --

# many rows of any alignment, in tiles of 32 or 64 rows and in copies
SIZES += [(2000, 777, 1001, 0, 0), (8000, 129, 300, 3, 1), (1500, 260, 2001, 0, 0), (1100, 2000, 259, 0, 0)]


@pytest.mark.parametrize("size", SIZES, ids=ids)
def test_linear_exact(size):
    M, N, K, pad, offset = size
    gen = generator(M * 7 + N * 3 + K)
    x, w = codes(gen, M, K, 3, pad, offset), codes(gen, N, K, 3, pad, offset)
    xs, ws = powers(gen, M), powers(gen, N)
    b, r = whole(gen, 1, N, 8)[0], whole(gen, M, N, 8, pad, offset)
    out = Out(M, N, F, pad, offset)
    T.taco_linear_int8(x, xs, w, ws, out.t, bias=b, act=RELU, residual=r,
                       workspace=space(T.taco_linear_int8_workspace_bytes(M, N, K)))
    torch.cuda.synchronize()
    out.check("out")
    z = (x.double() @ w.double().t()) * xs.double()[:, None] * ws.double()
    assert torch.equal(out.t.double(), (z + b.double()).clamp(min=0) + r.double())
    plain = Out(M, N, BF, pad, offset)
    T.taco_linear_int8(x, xs, w, ws, plain.t, workspace=space(T.taco_linear_int8_workspace_bytes(M, N, K)))
    torch.cuda.synchronize()
    plain.check("plain")
    assert torch.equal(plain.t, z.to(BF))


@pytest.mark.parametrize("size", SIZES, ids=ids)
def test_gated_exact(size):
    M, N, K, pad, offset = size
    gen = generator(M * 5 + N * 2 + K)
    x, w = codes(gen, M, K, 1, pad, offset), codes(gen, 2 * N, K, 1, pad, offset)
    xs, ws = torch.exp2(torch.randint(-1, 2, (M,), generator=gen, device=DEV).float()), powers(gen, 2 * N)
    out = Out(M, N, F, pad, offset)
    T.taco_gated_linear_int8(x, xs, w, ws, out.t, act=RELU,
                             workspace=space(T.taco_gated_linear_int8_workspace_bytes(M, N, K)))
    torch.cuda.synchronize()
    out.check("out")
    z = (x.double() @ w.double().t()) * xs.double()[:, None] * ws.double()
    assert torch.equal(out.t.double(), z[:, :N].clamp(min=0) * z[:, N:])


# large tiles with K whole and cut, in place and packed, as in test_layers_large.py with twice the K
@pytest.mark.parametrize("size", [(4100, 4104, 4112, 0, 0), (4090, 4090, 2000, 0, 0), (4099, 4101, 4115, 3, 0)], ids=ids)
def test_large_tiles(size):
    M, N, K, pad, _ = size
    gen = generator(M + N + K)
    x, w = codes(gen, M, K, 3, pad), codes(gen, N, K, 3, pad)
    xs, ws, b = powers(gen, M), powers(gen, N), whole(gen, 1, N, 8)[0]
    want = (x.double() @ w.double().t()) * xs.double()[:, None] * ws.double() + b.double()
    out = Out(M, N, F, pad)
    T.taco_linear_int8(x, xs, w, ws, out.t, bias=b, workspace=space(T.taco_linear_int8_workspace_bytes(M, N, K)))
    half = Out(M, N // 2, F, pad)
    hs = torch.exp2(torch.randint(-1, 1, (M,), generator=gen, device=DEV).float())
    wide = w[:N // 2 * 2]
    T.taco_gated_linear_int8(x.clamp(-1, 1), hs, wide.clamp(-1, 1), ws[:N // 2 * 2].contiguous(), half.t, act=RELU,
                             workspace=space(T.taco_gated_linear_int8_workspace_bytes(M, N // 2, K)))
    torch.cuda.synchronize()
    out.check("out")
    half.check("gated")
    assert torch.equal(out.t.double(), want)
    z = (x.clamp(-1, 1).double() @ wide.clamp(-1, 1).double().t()) * hs.double()[:, None] * ws[:N // 2 * 2].double()
    assert torch.equal(half.t.double(), z[:, :N // 2].clamp(min=0) * z[:, N // 2:])


# about where rows stop being few: the same sizes in rows of codes and of pairs
# of them, copied, and where they lie
@pytest.mark.parametrize("pad", [0, 16, 3])
@pytest.mark.parametrize("M,N,K", [(64, 4096, 4096), (64, 4096, 4112), (64, 4096, 8192), (33, 8192, 4096), (5, 16384, 16384)])
def test_where_rows_stop_being_few(M, N, K, pad):
    gen = generator(M + N + K)
    x, w = codes(gen, M, K, 3, pad), codes(gen, N, K, 3, pad)
    xs, ws = powers(gen, M), powers(gen, N)
    out, half = Out(M, N, F), Out(M, N // 2, F)
    T.taco_linear_int8(x, xs, w, ws, out.t, workspace=space(T.taco_linear_int8_workspace_bytes(M, N, K)))
    T.taco_gated_linear_int8(x, xs, w, ws, half.t, act=NONE, workspace=space(T.taco_gated_linear_int8_workspace_bytes(M, N // 2, K)))
    torch.cuda.synchronize()
    out.check("out")
    half.check("gated")
    z = (x.double() @ w.double().t()) * xs.double()[:, None] * ws.double()
    assert torch.equal(out.t.double(), z)
    want = z[:, :N // 2] * z[:, N // 2:]
    within(half.t, want, U32 * want.abs(), "gated")


@pytest.mark.parametrize("M,N", [(1, 16), (3, 40), (130, 260)])
def test_largest_sums(M, N):
    """-128 times -128 over the longest K: 131071 * 2^14, the largest sum that 32
    bits hold; and its negative, 127 * -128 * K."""
    K = T.TACO_INT8_MAX_K
    x = torch.full((M, K), -128, dtype=torch.int8, device=DEV)
    w = torch.full((N, K), -128, dtype=torch.int8, device=DEV)
    w[1::2] = 127
    one = torch.ones(max(M, N), device=DEV)
    out = Out(M, N, F)
    T.taco_linear_int8(x, one[:M], w, one[:N], out.t, workspace=space(T.taco_linear_int8_workspace_bytes(M, N, K)))
    torch.cuda.synchronize()
    out.check("out")
    want = torch.full((M, N), K * 2 ** 14, dtype=torch.float64, device=DEV)
    want[:, 1::2] = float(np.float32(-128 * 127 * K))
    assert torch.equal(out.t.double(), want)


@pytest.mark.parametrize("bias,residual,out", [(F, F, F), (BF, F, BF), (F, BF, F)])
@pytest.mark.parametrize("size", [(2, 40, 128), (128, 256, 256), (130, 260, 256), (3584, 3840, 128), (3600, 3604, 144)])
def test_epilogue_types(size, bias, residual, out):
    M, N, K = size
    gen = generator(M + N + K)
    x, w = codes(gen, M, K, 1), codes(gen, N, K, 1)
    xs, ws = powers(gen, M), powers(gen, N)
    b, r = whole(gen, 1, N, 8, dtype=bias)[0], whole(gen, M, N, 8, dtype=residual)
    o = Out(M, N, out)
    T.taco_linear_int8(x, xs, w, ws, o.t, bias=b, act=RELU, residual=r,
                       workspace=space(T.taco_linear_int8_workspace_bytes(M, N, K)))
    torch.cuda.synchronize()
    o.check("out")
    z = (x.double() @ w.double().t()) * xs.double()[:, None] * ws.double() + b.double()
    assert torch.equal(o.t, (z.clamp(min=0) + r.double()).to(out))


# ------------------------------------------------------------- real values --

REAL = [(1, 264, 520, 0, 0), (3, 100, 333, 1, 0), (24, 328, 1000, 0, 0), (40, 520, 1024, 0, 0), (130, 264, 2056, 8, 0),
        (300, 516, 700, 0, 0), (600, 520, 264, 3, 1), (513, 1024, 1040, 16, 0)]


def real_codes(gen, M, N, K, pad, offset):
    x, w = codes(gen, M, K, 127, pad, offset), codes(gen, N, K, 127, pad, offset)
    xs = torch.rand(M, generator=gen, device=DEV) * 0.02 + 0.01
    ws = (torch.rand(N, generator=gen, device=DEV) + 0.5) / (40 * math.sqrt(K))
    z = (x.double() @ w.double().t()) * xs.double()[:, None] * ws.double()
    return x, xs, w, ws, z


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("size", REAL, ids=ids)
def test_linear_real(size, act):
    M, N, K, pad, offset = size
    gen = generator(M + N + K + act)
    x, xs, w, ws, z = real_codes(gen, M, N, K, pad, offset)
    b, r = matrix(gen, 1, N, F)[0], matrix(gen, M, N, BF, pad)
    tz = 4 * U32 * z.abs() + U32 * b.double().abs()
    z = z + b.double()
    for od in (BF, F):
        out = Out(M, N, od, pad, offset)
        T.taco_linear_int8(x, xs, w, ws, out.t, bias=b, act=act, residual=r,
                           workspace=space(T.taco_linear_int8_workspace_bytes(M, N, K)))
        torch.cuda.synchronize()
        out.check("out")
        want = act64(z, act) + r.double()
        t = 1.13 * tz + 32 * U32 * z.abs() + U32 * (want.abs() + r.double().abs())
        within(out.t, want, t + UNIT[od] * (want.abs() + t), "out")


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("size", REAL, ids=ids)
def test_gated_real(size, act):
    M, N, K, pad, offset = size
    gen = generator(M + N + K + act)
    x, xs, w, ws, z = real_codes(gen, M, 2 * N, K, pad, offset)
    tz = 4 * U32 * z.abs()
    for od in (BF, F):
        out = Out(M, N, od, pad, offset)
        T.taco_gated_linear_int8(x, xs, w, ws, out.t, act=act,
                                 workspace=space(T.taco_gated_linear_int8_workspace_bytes(M, N, K)))
        torch.cuda.synchronize()
        out.check("out")
        v, u = act64(z[:, :N], act), z[:, N:]
        tv = 1.13 * tz[:, :N] + 32 * U32 * z[:, :N].abs()
        want = v * u
        t = tv * u.abs() + v.abs() * tz[:, N:] + tv * tz[:, N:] + U32 * want.abs()
        within(out.t, want, t + UNIT[od] * (want.abs() + t), "out")


# ----------------------------------------------------------------- the rest --

def test_a_rows_nan_stays_in_it():
    """Quantised and multiplied: rows of x and w with an infinity or NaN give NaN
    in their row and column, and the others' bits stay."""
    gen = generator(3)
    M, N, K = 150, 140, 304
    x, w = matrix(gen, M, K, BF), matrix(gen, N, K, BF)
    outs = []
    for bad in (False, True):
        if bad:
            x[7, 3], x[149, 0], w[20, 303] = math.inf, math.nan, -math.inf
        qx, qw = (torch.empty(n, K, dtype=torch.int8, device=DEV) for n in (M, N))
        xs, ws = torch.empty(M, device=DEV), torch.empty(N, device=DEV)
        T.taco_quantize_rows(x, qx, xs)
        T.taco_quantize_rows(w, qw, ws)
        out = torch.empty(M, N, device=DEV)
        T.taco_linear_int8(qx, xs, qw, ws, out, act=SILU, workspace=space(T.taco_linear_int8_workspace_bytes(M, N, K)))
        outs.append(out)
    torch.cuda.synchronize()
    fine_r = torch.ones(M, dtype=torch.bool, device=DEV)
    fine_c = torch.ones(N, dtype=torch.bool, device=DEV)
    fine_r[[7, 149]], fine_c[20] = False, False
    assert torch.equal(outs[0][fine_r][:, fine_c], outs[1][fine_r][:, fine_c])
    assert bool(torch.isnan(outs[1][~fine_r]).all()) and bool(torch.isnan(outs[1][:, ~fine_c]).all())


def test_no_rows():
    w, ws = torch.zeros(24, 40, dtype=torch.int8, device=DEV), torch.ones(24, device=DEV)
    x, xs = torch.empty(0, 40, dtype=torch.int8, device=DEV), torch.empty(0, device=DEV)
    T.taco_quantize_rows(torch.empty(0, 40, device=DEV), x, xs)
    T.taco_linear_int8(x, xs, w, ws, torch.empty(0, 24, device=DEV))
    T.taco_gated_linear_int8(x, xs, w, ws, torch.empty(0, 12, device=DEV))
    torch.cuda.synchronize()


@pytest.mark.parametrize("M", [3, 24, 300])
def test_other_stream_and_graph(M):
    """Rows quantised and multiplied twice (a gated feed-forward) on a stream of
    its own, then captured and replayed with other inputs."""
    gen = generator(M)
    H, I = 272, 520
    x = matrix(gen, M, H, BF)
    w1, w2 = matrix(gen, 2 * I, H, BF, sigma=0.1), matrix(gen, H, I, BF, sigma=0.1)
    q1, q2 = (torch.empty(*w.shape, dtype=torch.int8, device=DEV) for w in (w1, w2))
    s1, s2 = torch.empty(2 * I, device=DEV), torch.empty(H, device=DEV)
    qx, qh = torch.empty(M, H, dtype=torch.int8, device=DEV), torch.empty(M, I, dtype=torch.int8, device=DEV)
    sx, sh = torch.empty(M, device=DEV), torch.empty(M, device=DEV)
    h, y = torch.empty(M, I, device=DEV), torch.empty(M, H, device=DEV)
    ws1 = space(T.taco_gated_linear_int8_workspace_bytes(M, I, H))
    ws2 = space(T.taco_linear_int8_workspace_bytes(M, H, I))

    def layer():
        T.taco_quantize_rows(x, qx, sx)
        T.taco_gated_linear_int8(qx, sx, q1, s1, h, workspace=ws1)
        T.taco_quantize_rows(h, qh, sh)
        T.taco_linear_int8(qh, sh, q2, s2, y, residual=x, workspace=ws2)

    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        T.taco_quantize_rows(w1, q1, s1)
        T.taco_quantize_rows(w2, q2, s2)
        layer()
    stream.synchronize()
    eager = y.clone()
    z = (qx.double() @ q1.double().t()) * sx.double()[:, None] * s1.double()
    tz = 4 * U32 * z.abs()
    v, u = act64(z[:, :I], SILU), z[:, I:]
    tv = 1.13 * tz[:, :I] + 32 * U32 * z[:, :I].abs()
    within(h, v * u, tv * u.abs() + v.abs() * tz[:, I:] + tv * tz[:, I:] + 2 * U32 * (v * u).abs(), "h")
    out = (qh.double() @ q2.double().t()) * sh.double()[:, None] * s2.double()
    within(y, out + x.double(), 4 * U32 * out.abs() + 2 * U32 * (out + x.double()).abs(), "y")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer()
    for k in range(4):
        x.copy_(matrix(generator(k), M, H, BF) if k else x)
        graph.replay()
        torch.cuda.synchronize()
        got = y.clone()
        layer()
        torch.cuda.synchronize()
        assert torch.equal(got, y)
        if k == 0:
            assert torch.equal(got, eager)
