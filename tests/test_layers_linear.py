"""The projections, plain and gated, forward and backward, against their
formulas in float64.

Two kinds of checks. With small whole numbers every product and sum is exact in
float32, so a float32 output must equal the definition: this is what finds an
index, a mask or a split that is wrong, at every edge. With normal values the
outputs lie within what float32 sums and the stated roundings allow:
  sums     each 16 products enter the accumulator with at most four roundings,
           parts of a sum are joined with one each: (K / 4 + 64) U32 times the
           sum of magnitudes
  act      at most 32 U32 of |t| for a value (|act'| <= 1.13 on what comes in),
           64 U32 for a slope: a few units of exp, erf and the steps between,
           and exp's argument, t or t^2 / 2, to one unit
  dz       its rounding to bf16, 2^-8
  stores   U32 or 2^-8"""

import math

import pytest
import torch

import quantized_compression_tensor_amd as T
from tests.layers_util import DEV, U32, UNIT, Out, generator, matrix, within

pytestmark = pytest.mark.gpu

BF, F = torch.bfloat16, torch.float32
NONE, GELU, SILU, RELU = T.TACO_ACT_NONE, T.TACO_ACT_GELU, T.TACO_ACT_SILU, T.TACO_ACT_RELU
ACTS = [NONE, GELU, SILU, RELU]

# (M, N, K, pad, offset): edges of tiles, single rows, columns and k, rows that
# start anywhere, few tiles with a long K, many tiles
SIZES = [
    (1, 1, 1, 0, 0), (1, 8, 8, 0, 0), (1, 64, 64, 0, 0), (1, 7, 9, 1, 1), (2, 3, 65, 3, 1), (1, 4096, 512, 0, 0),
    (1, 1000, 4104, 0, 0), (1, 1001, 4099, 5, 3), (4, 640, 1536, 8, 0), (5, 77, 2050, 0, 1), (15, 16, 32, 0, 0),
    (16, 512, 1024, 0, 0), (17, 33, 63, 1, 0), (24, 1728, 264, 0, 0), (31, 129, 257, 8, 8), (32, 256, 4096, 0, 0),
    (33, 128, 128, 0, 0), (48, 1024, 8192, 0, 0), (63, 64, 72, 0, 0), (64, 65, 1000, 3, 3), (100, 300, 500, 8, 8),
    (127, 128, 64, 0, 0), (128, 128, 128, 0, 0), (129, 127, 129, 1, 1), (200, 520, 192, 24, 16), (255, 257, 320, 0, 0),
    (256, 256, 256, 0, 0), (257, 264, 328, 0, 8), (300, 1032, 1288, 0, 0), (512, 512, 4096, 0, 0),
    (511, 515, 1021, 3, 0), (768, 768, 512, 8, 0), (1001, 777, 1285, 3, 1), (2048, 2048, 256, 0, 0),
    (1500, 1480, 6000, 0, 0), (3000, 1100, 136, 4, 4), (4100, 4104, 72, 0, 0), (70000, 24, 16, 0, 0), (130, 60008, 24, 0, 0),
]


def ids(s):
    return "x".join(map(str, s[:3])) + f"-p{s[3]}o{s[4]}"


def act64(t, act):
    if act == GELU:
        return t * torch.special.ndtr(t)
    if act == SILU:
        return t * torch.sigmoid(t)
    return t.clamp(min=0) if act == RELU else t


def slope64(t, act):
    if act == GELU:
        return torch.special.ndtr(t) + t * torch.exp(-t * t / 2) / math.sqrt(2 * math.pi)
    if act == SILU:
        s = torch.sigmoid(t)
        return s + t * s * (1 - s)
    return (t > 0).double() if act == RELU else torch.ones_like(t)


def whole(gen, rows, cols, most, pad=0, offset=0, dtype=BF):
    m = matrix(gen, rows, cols, dtype, pad, offset)
    return m.copy_(torch.randint(-most, most + 1, (rows, cols), generator=gen, device=DEV))


def space(n):
    return torch.empty(n, dtype=torch.uint8, device=DEV).fill_(0xFF) if n else None


def product64(a, b):
    """a b^T and the sum of magnitudes, in float64."""
    a, b = a.double(), b.double()
    return a @ b.t(), a.abs() @ b.abs().t()


# ---------------------------------------------------------------- exactly --

@pytest.mark.parametrize("size", SIZES, ids=ids)
def test_linear_exact(size):
    M, N, K, pad, offset = size
    gen = generator(M * 7 + N * 3 + K)
    x, w = whole(gen, M, K, 3, pad, offset), whole(gen, N, K, 3, pad, offset)
    b, r = whole(gen, 1, N, 8)[0], whole(gen, M, N, 8, pad, offset)
    out, z = Out(M, N, F, pad, offset), Out(M, N, F, pad, offset)
    T.taco_linear(x, w, out.t, bias=b, act=RELU, residual=r, preact=z.t,
                  workspace=space(T.taco_linear_workspace_bytes(M, N, K)))
    torch.cuda.synchronize()
    out.check("out")
    z.check("preact")
    want = x.double() @ w.double().t() + b.double()
    assert torch.equal(z.t.double(), want)
    assert torch.equal(out.t.double(), want.clamp(min=0) + r.double())
    plain = Out(M, N, BF, pad, offset)
    T.taco_linear(x, w, plain.t, workspace=space(T.taco_linear_workspace_bytes(M, N, K)))
    torch.cuda.synchronize()
    plain.check("plain")
    assert torch.equal(plain.t, (x.double() @ w.double().t()).to(BF))


@pytest.mark.parametrize("bias,residual,out", [(F, F, F), (BF, F, BF), (F, BF, F)])
@pytest.mark.parametrize("size", [(2, 40, 64), (128, 256, 128), (130, 260, 128), (3584, 3840, 64), (3600, 3604, 72)])
def test_epilogue_types(size, bias, residual, out):
    """Tiles with and without an edge, of either size, in each element type."""
    M, N, K = size
    gen = generator(M + N + K)
    x, w = whole(gen, M, K, 1), whole(gen, N, K, 1)
    b, r = whole(gen, 1, N, 8, dtype=bias)[0], whole(gen, M, N, 8, dtype=residual)
    o, z = Out(M, N, out), Out(M, N, out)
    T.taco_linear(x, w, o.t, bias=b, act=RELU, residual=r, preact=z.t,
                  workspace=space(T.taco_linear_workspace_bytes(M, N, K)))
    torch.cuda.synchronize()
    o.check("out")
    z.check("preact")
    want = x.double() @ w.double().t() + b.double()
    assert torch.equal(z.t, want.to(out))
    assert torch.equal(o.t, (want.clamp(min=0) + r.double()).to(out))


@pytest.mark.parametrize("size", SIZES, ids=ids)
def test_gated_exact(size):
    M, N, K, pad, offset = size
    gen = generator(M * 5 + N * 2 + K)
    x, w = whole(gen, M, K, 1, pad, offset), whole(gen, 2 * N, K, 1, pad, offset)
    out, z = Out(M, N, F, pad, offset), Out(M, 2 * N, F, pad, offset)
    T.taco_gated_linear(x, w, out.t, act=RELU, preact=z.t,
                        workspace=space(T.taco_gated_linear_workspace_bytes(M, N, K)))
    torch.cuda.synchronize()
    out.check("out")
    z.check("preact")
    want = x.double() @ w.double().t()
    assert torch.equal(z.t.double(), want)
    assert torch.equal(out.t.double(), want[:, :N].clamp(min=0) * want[:, N:])


@pytest.mark.parametrize("size", SIZES, ids=ids)
def test_linear_backward_exact(size):
    """No activation, and relu with a whole dout, whose dz is exact in bf16."""
    M, N, K, pad, offset = size
    gen = generator(M * 3 + N + K)
    x, w = whole(gen, M, K, 3, pad, offset), whole(gen, N, K, 3, pad, offset)
    d, z = whole(gen, M, N, 3, pad, offset), whole(gen, M, N, 2, pad, offset)
    for act in (NONE, RELU):
        dx, dw, db = Out(M, K, F, pad, offset), Out(N, K, F, pad, offset), Out(1, N, F)
        T.taco_linear_backward(d, x, w, act=act, preact=z if act else None, dx=dx.t, dw=dw.t, dbias=db.vector(),
                               workspace=space(T.taco_linear_backward_workspace_bytes(M, N, K)))
        torch.cuda.synchronize()
        for o, n in ((dx, "dx"), (dw, "dw"), (db, "dbias")):
            o.check(n)
        dz = d.double() * slope64(z.double(), act)
        assert torch.equal(dx.t.double(), dz @ w.double()), act
        assert torch.equal(dw.t.double(), dz.t() @ x.double()), act
        assert torch.equal(db.vector().double(), dz.sum(0)), act


@pytest.mark.parametrize("size", SIZES, ids=ids)
def test_gated_backward_exact(size):
    M, N, K, pad, offset = size
    gen = generator(M * 2 + N + K)
    x, w = whole(gen, M, K, 2, pad, offset), whole(gen, 2 * N, K, 2, pad, offset)
    d, z = whole(gen, M, N, 2, pad, offset), whole(gen, M, 2 * N, 2, pad, offset, F)
    dx, dw = Out(M, K, F, pad, offset), Out(2 * N, K, BF, pad, offset)
    T.taco_gated_linear_backward(d, x, w, act=RELU, preact=z, dx=dx.t, dw=dw.t,
                                 workspace=space(T.taco_gated_linear_backward_workspace_bytes(M, N, K)))
    torch.cuda.synchronize()
    dx.check("dx")
    dw.check("dw")
    d64, g, u = d.double(), z[:, :N].double(), z[:, N:].double()
    dz = torch.cat([d64 * u * slope64(g, RELU), d64 * act64(g, RELU)], 1)
    assert torch.equal(dx.t.double(), dz @ w.double())
    assert torch.equal(dw.t, (dz.t() @ x.double()).to(BF))


# ------------------------------------------------------------ real values --

REAL = [(1, 264, 520, 0, 0), (3, 100, 333, 1, 0), (40, 520, 1024, 0, 0), (130, 264, 2056, 8, 0), (300, 516, 700, 0, 0),
        (600, 520, 264, 3, 1), (513, 1024, 1032, 0, 0)]


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("size", REAL, ids=ids)
def test_linear_real(size, act):
    M, N, K, pad, offset = size
    gen = generator(M + N + K + act)
    x, w = matrix(gen, M, K, BF, pad, offset), matrix(gen, N, K, BF, pad, offset, sigma=3 / math.sqrt(K))
    b, r = matrix(gen, 1, N, F)[0], matrix(gen, M, N, BF, pad)
    for od, zd in ((BF, F), (F, BF)):
        out, zo = Out(M, N, od, pad, offset), Out(M, N, zd)
        T.taco_linear(x, w, out.t, bias=b, act=act, residual=r, preact=zo.t,
                      workspace=space(T.taco_linear_workspace_bytes(M, N, K)))
        torch.cuda.synchronize()
        out.check("out")
        zo.check("preact")
        z, size_ = product64(x, w)
        z = z + b.double()
        tz = (K / 4 + 64) * U32 * (size_ + b.double().abs())
        within(zo.t, z, tz + UNIT[zd] * (z.abs() + tz), "preact")
        want = act64(z, act) + r.double()
        t = 1.13 * tz + 32 * U32 * z.abs() + U32 * (want.abs() + r.double().abs())
        within(out.t, want, t + UNIT[od] * (want.abs() + t), "out")


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("size", REAL, ids=ids)
def test_gated_real(size, act):
    M, N, K, pad, offset = size
    gen = generator(M + N + K + act)
    x, w = matrix(gen, M, K, BF, pad, offset), matrix(gen, 2 * N, K, BF, pad, offset, sigma=3 / math.sqrt(K))
    for od, zd in ((BF, F), (F, BF)):
        out, zo = Out(M, N, od, pad, offset), Out(M, 2 * N, zd)
        T.taco_gated_linear(x, w, out.t, act=act, preact=zo.t,
                            workspace=space(T.taco_gated_linear_workspace_bytes(M, N, K)))
        torch.cuda.synchronize()
        out.check("out")
        zo.check("preact")
        z, size_ = product64(x, w)
        tz = (K / 4 + 64) * U32 * size_
        within(zo.t, z, tz + UNIT[zd] * (z.abs() + tz), "preact")
        v, u = act64(z[:, :N], act), z[:, N:]
        tv = 1.13 * tz[:, :N] + 32 * U32 * z[:, :N].abs()
        want = v * u
        t = tv * u.abs() + v.abs() * tz[:, N:] + tv * tz[:, N:] + U32 * want.abs()
        within(out.t, want, t + UNIT[od] * (want.abs() + t), "out")


def check_gradients(dz, tdz, x, w, dx, dw, M, wide):
    """dx and dw from dz in float64, of which the kernel's operand is tdz off."""
    for got, a, ta, b, n, what in ((dx, dz, tdz, w.t(), wide, "dx"), (dw, dz.t(), tdz.t(), x.t(), M, "dw")):
        want, size = product64(a, b)
        t = ta @ b.double().abs().t() + (n / 4 + 64) * U32 * (size + ta @ b.double().abs().t())
        within(got, want, t + UNIT[got.dtype] * (want.abs() + t), what)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("size", REAL, ids=ids)
def test_linear_backward_real(size, act):
    M, N, K, pad, offset = size
    gen = generator(M + N + K + act)
    x, w = matrix(gen, M, K, BF, pad, offset), matrix(gen, N, K, BF, pad, offset, sigma=0.1)
    for zd, gd in ((BF, BF), (F, F)):
        d, z = matrix(gen, M, N, BF, pad), matrix(gen, M, N, zd, pad, sigma=2.0)
        dx, dw, db = Out(M, K, gd, pad, offset), Out(N, K, gd), Out(1, N, F)
        T.taco_linear_backward(d, x, w, act=act, preact=z, dx=dx.t, dw=dw.t, dbias=db.vector(),
                               workspace=space(T.taco_linear_backward_workspace_bytes(M, N, K)))
        torch.cuda.synchronize()
        for o, n in ((dx, "dx"), (dw, "dw"), (db, "dbias")):
            o.check(n)
        dz = d.double() * slope64(z.double(), act)
        t32 = torch.zeros_like(dz) if act == NONE else 64 * U32 * d.double().abs()
        check_gradients(dz, t32 + (0 if act == NONE else 2.0 ** -8) * (dz.abs() + t32), x, w, dx.t, dw.t, M, N)
        within(db.vector(), dz.sum(0), t32.sum(0) + (M / 4 + 64) * U32 * (dz.abs() + t32).sum(0)
               + U32 * dz.sum(0).abs(), "dbias")


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("size", REAL, ids=ids)
def test_gated_backward_real(size, act):
    M, N, K, pad, offset = size
    gen = generator(M + N + K + act)
    x, w = matrix(gen, M, K, BF, pad, offset), matrix(gen, 2 * N, K, BF, pad, offset, sigma=0.1)
    for zd, gd in ((BF, BF), (F, F)):
        d, z = matrix(gen, M, N, BF, pad), matrix(gen, M, 2 * N, zd, pad, sigma=2.0)
        dx, dw = Out(M, K, gd, pad, offset), Out(2 * N, K, gd)
        T.taco_gated_linear_backward(d, x, w, act=act, preact=z, dx=dx.t, dw=dw.t,
                                     workspace=space(T.taco_gated_linear_backward_workspace_bytes(M, N, K)))
        torch.cuda.synchronize()
        dx.check("dx")
        dw.check("dw")
        d64, g, u = d.double(), z[:, :N].double(), z[:, N:].double()
        dz = torch.cat([d64 * u * slope64(g, act), d64 * act64(g, act)], 1)
        t32 = torch.cat([66 * U32 * (d64 * u).abs(), 34 * U32 * (d64 * g).abs()], 1)
        check_gradients(dz, t32 + 2.0 ** -8 * (dz.abs() + t32), x, w, dx.t, dw.t, M, 2 * N)


# ------------------------------------------------------------- activations --

@pytest.mark.parametrize("act", ACTS)
def test_activations_over_their_range(act):
    """Value and slope from -110 to 110, at infinities and NaN: z is one
    product with 1, so out is act(z) alone."""
    t = torch.cat([torch.linspace(-110, 110, 1981), torch.linspace(-1e-3, 1e-3, 57),
                   torch.tensor([0.0, -0.0, 1e-30, -1e-30, 3e38, -3e38, math.inf, -math.inf, math.nan])]).to(DEV, BF)
    n = t.numel()
    x, w = t.view(n, 1).contiguous(), torch.ones(1, 1, dtype=BF, device=DEV)
    out = torch.empty(n, 1, device=DEV)
    T.taco_linear(x, w, out, act=act, workspace=space(T.taco_linear_workspace_bytes(n, 1, 1)))
    d = torch.ones(n, 1, dtype=BF, device=DEV)
    dx = torch.empty(n, 1, device=DEV)
    T.taco_linear_backward(d, x, w, act=act, preact=x, dx=dx,
                           workspace=space(T.taco_linear_backward_workspace_bytes(n, 1, 1)))
    torch.cuda.synchronize()
    t64 = t.double()[:, None]
    v, s = act64(t64, act), slope64(t64, act)
    odd = ~torch.isfinite(t64)
    # at the infinities the formulas give inf, nan or a limit: any of the latter two for -inf
    assert bool(torch.isnan(out[torch.isnan(t64)]).all())
    assert bool((out[t64 == math.inf] == math.inf).all())
    low = out[t64 == -math.inf]
    assert bool((torch.isnan(low) | (low == (-math.inf if act == NONE else 0.0))).all())
    within(out[~odd], v[~odd], 32 * U32 * t64[~odd].abs() + U32 * v[~odd].abs(), "value")
    fine = ~odd & (t64.abs() < 1e18)      # beyond, t^2 is not finite in float32
    within(dx[fine], s[fine], 64 * U32 + 2.0 ** -8 * (s[fine].abs() + 64 * U32), "slope")


def test_nonfinite_values_stay_in_their_rows():
    """A row of x with an infinity or NaN leaves the other rows' bits alone,
    and what lies between the rows of any operand never enters (it is NaN in
    every test here)."""
    gen = generator(11)
    M, N, K = 200, 300, 328
    x, w = matrix(gen, M, K, BF), matrix(gen, N, K, BF)
    clean = torch.empty(M, N, device=DEV)
    ws = space(T.taco_linear_workspace_bytes(M, N, K))
    T.taco_linear(x, w, clean, act=GELU, workspace=ws)
    bad = x.clone()
    bad[7, 5], bad[130, 327], bad[199, 0] = math.inf, math.nan, -math.inf
    out = torch.empty(M, N, device=DEV)
    T.taco_linear(bad, w, out, act=GELU, workspace=ws)
    torch.cuda.synchronize()
    rows = torch.ones(M, dtype=torch.bool, device=DEV)
    rows[[7, 130, 199]] = False
    assert torch.equal(out[rows], clean[rows])
    assert not bool(torch.isfinite(out[130]).any())


# ----------------------------------------------------------------- the rest --

def test_no_rows():
    """M == 0: the forward calls do nothing, the backward calls clear dw and dbias."""
    x, w, e = torch.empty(0, 40, dtype=BF, device=DEV), torch.zeros(24, 40, dtype=BF, device=DEV), \
        torch.empty(0, 24, dtype=BF, device=DEV)
    T.taco_linear(x, w, e)
    T.taco_gated_linear(x, w, e[:, :12])
    dw, db = Out(24, 40, F), Out(1, 24, F)
    T.taco_linear_backward(e, x, w, act=GELU, preact=e, dx=torch.empty_like(x), dw=dw.t, dbias=db.vector(),
                           workspace=space(T.taco_linear_backward_workspace_bytes(0, 24, 40)))
    dg = Out(24, 40, BF)
    T.taco_gated_linear_backward(e[:, :12], x, w, preact=e, dx=torch.empty_like(x), dw=dg.t,
                                 workspace=space(T.taco_gated_linear_backward_workspace_bytes(0, 12, 40)))
    torch.cuda.synchronize()
    for o in (dw, db, dg):
        o.check("cleared")
        assert not o.t.any()


@pytest.mark.parametrize("parts", [("dx",), ("dw",), ("dbias",), ("dx", "dbias"), ("dw", "dbias")])
def test_backward_parts(parts):
    gen = generator(12)
    M, N, K = 70, 136, 200
    x, w, d, z = (matrix(gen, *s, BF) for s in ((M, K), (N, K), (M, N), (M, N)))
    full = {"dx": torch.empty(M, K, device=DEV), "dw": torch.empty(N, K, device=DEV), "dbias": torch.empty(N, device=DEV)}
    ws = space(T.taco_linear_backward_workspace_bytes(M, N, K))
    for act in (NONE, GELU):
        T.taco_linear_backward(d, x, w, act=act, preact=z, workspace=ws, **full)
        some = {p: torch.empty_like(full[p]) for p in parts}
        T.taco_linear_backward(d, x, w, act=act, preact=z, workspace=ws, **some)
        torch.cuda.synchronize()
        for p in parts:
            assert torch.equal(some[p], full[p]), p


def test_gradients_against_differences():
    """Directional derivatives of sum(out * c) with the forward formulas in
    float64, central differences of step 1e-4 (error below 1e-6 of the terms);
    the kernel's dz carries one bf16 rounding, 2^-8 of each of its terms."""
    gen = generator(13)
    M, N, K, h = 20, 24, 40, 1e-4
    x = matrix(gen, M, K, BF)
    c = matrix(gen, M, N, BF)
    for act in (GELU, SILU):
        for gated in (False, True):
            wide = 2 * N if gated else N
            w = matrix(gen, wide, K, BF, sigma=0.3)

            def forward(x_, w_):
                z = x_ @ w_.t()
                return act64(z[:, :N], act) * z[:, N:] if gated else act64(z, act)

            def loss(x_, w_):
                return float((forward(x_, w_) * c.double()).sum())

            z = (x.double() @ w.double().t()).float()
            dx, dw = torch.empty(M, K, device=DEV), torch.empty(wide, K, device=DEV)
            f = T.taco_gated_linear_backward if gated else T.taco_linear_backward
            size = (T.taco_gated_linear_backward_workspace_bytes if gated else T.taco_linear_backward_workspace_bytes)(M, N, K)
            f(c, x, w, act=act, preact=z, dx=dx, dw=dw, workspace=space(size))
            torch.cuda.synchronize()
            X, W = x.double(), w.double()
            # the sum of magnitudes that dz's rounding acts on
            zt = z.double().requires_grad_(True)
            o = act64(zt[:, :N], act) * zt[:, N:] if gated else act64(zt, act)
            (dz,) = torch.autograd.grad((o * c.double()).sum(), zt)
            for seed in range(2):
                g = generator(200 + seed)
                vx = torch.randn(M, K, generator=g, device=DEV).double()
                vw = torch.randn(wide, K, generator=g, device=DEV).double()
                for got, v, plus, minus, terms in (
                        (dx, vx, loss(X + h * vx, W), loss(X - h * vx, W), (dz.abs() @ W.abs() * vx.abs()).sum()),
                        (dw, vw, loss(X, W + h * vw), loss(X, W - h * vw), (dz.abs().t() @ X.abs() * vw.abs()).sum())):
                    assert abs(float((got.double() * v).sum()) - (plus - minus) / (2 * h)) <= (2.0 ** -8 + 1e-5) * float(terms)


def test_same_bits_streams_and_graphs():
    """The same call gives the same bits again, on a side stream, and captured
    in a graph and replayed on other inputs."""
    gen = generator(14)
    M, N, K = 160, 200, 1024
    sets = [[matrix(gen, M, K, BF), matrix(gen, N, K, BF, sigma=0.05), matrix(gen, M, N // 2, BF)] for _ in range(3)]
    ws_f = space(T.taco_gated_linear_workspace_bytes(M, N // 2, K))
    ws_b = space(T.taco_gated_linear_backward_workspace_bytes(M, N // 2, K))
    ws_l = space(T.taco_linear_workspace_bytes(M, K, N // 2))

    def buffers():
        return [torch.zeros(M, N // 2, dtype=BF, device=DEV), torch.zeros(M, N, dtype=BF, device=DEV),
                torch.zeros(M, K, dtype=BF, device=DEV), torch.zeros(N, K, device=DEV), torch.zeros(M, K, device=DEV)]

    def step(s, o, stream=None):
        T.taco_gated_linear(s[0], s[1], o[0], preact=o[1], workspace=ws_f, stream=stream)
        T.taco_gated_linear_backward(s[2], s[0], s[1], preact=o[1], dx=o[2], dw=o[3], workspace=ws_b, stream=stream)
        T.taco_linear(o[0], s[1].view(N * K)[:K * (N // 2)].view(K, N // 2), o[4], act=GELU, workspace=ws_l, stream=stream)

    eager = []
    for s in sets:
        o = buffers()
        step(s, o)
        torch.cuda.synchronize()
        eager.append(o)
    side = torch.cuda.Stream()
    o = buffers()
    torch.cuda.synchronize()
    step(sets[0], o, side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(o, eager[0]))
    live, o = [t.clone() for t in sets[0]], buffers()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step(live, o, side)
    for i in (1, 0, 2):
        for a, b in zip(live, sets[i]):
            a.copy_(b)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(o, eager[i])), i


def test_offsets_beyond_32_bits():
    """Rows that reach past 2^31 elements (and 2^32 bytes) of their tensor:
    2^20 rows 2104 elements apart. Whole numbers: exact, the sums over a
    million rows included."""
    M, N, K, apart = (1 << 20) + 37, 24, 40, 2104
    gen = generator(15)

    def far(cols, dtype=BF):
        return torch.empty(M * apart, dtype=dtype, device=DEV).view(M, apart)[:, :cols]

    x, d = far(K), far(N)
    x.copy_(torch.randint(-1, 2, (M, K), generator=gen, device=DEV))
    d.copy_(torch.randint(-1, 2, (M, N), generator=gen, device=DEV))
    w = whole(gen, N, K, 2)
    out, dx = far(N), far(K)
    T.taco_linear(x, w, out, workspace=space(T.taco_linear_workspace_bytes(M, N, K)))
    dw, db = torch.empty(N, K, device=DEV), torch.empty(N, device=DEV)
    T.taco_linear_backward(d, x, w, dx=dx, dw=dw, dbias=db,
                           workspace=space(T.taco_linear_backward_workspace_bytes(M, N, K)))
    torch.cuda.synchronize()
    x64, d64 = x.double(), d.double()
    assert torch.equal(out.double(), x64 @ w.double().t())
    assert torch.equal(dx.double(), d64 @ w.double())
    assert torch.equal(dw.double(), d64.t() @ x64)
    assert torch.equal(db.double(), d64.sum(0))
    y = far(K)
    T.taco_layer_norm(x, None, None, 1e-5, y)
    torch.cuda.synchronize()
    want = torch.nn.functional.layer_norm(x64[-1000:], (K,))
    within(y[-1000:], want, 2.0 ** -8 * want.abs() + 1e-4, "norm")
