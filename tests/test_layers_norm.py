"""Layer norm, forward and backward, against its formulas in float64.

Tolerances: a sum of `cols` float32 terms is formed from at most 8 * 4 serial
adds per lane, 6 between lanes and 16 between waves, so its error is below
64 U32 times the sum of magnitudes; the elementwise steps add a few U32 of
their terms. 128 U32 times the magnitudes that enter an element covers both;
a stored bf16 adds half a unit in the last place. Sums over rows: one add for
each row a workgroup takes and at most 160 between workgroups."""

import itertools

import pytest
import torch

import quantized_compression_tensor_amd as T
from tests.layers_util import DEV, U32, UNIT, Out, generator, matrix, within

pytestmark = pytest.mark.gpu

BF, F = torch.bfloat16, torch.float32
WIDTHS = [1, 2, 7, 8, 100, 128, 129, 256, 257, 500, 512, 513, 1025, 4096, 5120, 8191, 8192, 8193, 12001, 16379, 16384]
EPS = 1e-5


def forward64(x, weight, bias, eps):
    x = x.double()
    mean = x.mean(1, keepdim=True)
    d = x - mean
    rstd = 1 / torch.sqrt((d * d).mean(1, keepdim=True) + eps)
    y = d * rstd
    w = 1.0 if weight is None else weight.double()
    b = 0.0 if bias is None else bias.double()
    return y * w + b, mean[:, 0], rstd[:, 0]


def check_forward(x, weight, bias, eps, y_dtype, pad, offset, what):
    rows, cols = x.shape
    y, mean, rstd = Out(rows, cols, y_dtype, pad, offset), Out(1, rows, F), Out(1, rows, F)
    T.taco_layer_norm(x, weight, bias, eps, y.t, mean=mean.vector(), rstd=rstd.vector())
    torch.cuda.synchronize()
    for o, n in ((y, "y"), (mean, "mean"), (rstd, "rstd")):
        o.check(f"{what} {n}")
    wy, wm, wr = forward64(x, weight, bias, eps)
    x64 = x.double()
    size = x64.abs().mean(1)
    within(mean.vector(), wm, 128 * U32 * size, f"{what} mean")
    # rstd: the differences carry the mean's error, of first order only through
    # their sum, which is zero; second-order terms are covered by size^2 * wr^2
    within(rstd.vector(), wr, (128 * U32 + (128 * U32 * size * wr) ** 2) * wr, f"{what} rstd")
    w = torch.ones(cols, device=DEV).double() if weight is None else weight.double().abs()
    b = torch.zeros(cols, device=DEV).double() if bias is None else bias.double().abs()
    xhat = ((x64 - wm[:, None]) * wr[:, None]).abs()
    moved = 128 * U32 * ((xhat + (size * wr)[:, None]) * w + b)
    within(y.t, wy, moved + UNIT[y_dtype] * (wy.abs() + moved), f"{what} y")


@pytest.mark.parametrize("cols", WIDTHS)
def test_forward_widths(cols):
    for n, (xd, yd) in enumerate([(BF, BF), (F, BF), (F, F), (BF, F)]):
        gen = generator(cols * 10 + n)
        for rows, pad, offset in [(1, 0, 0), (3, 3, 1), (37, 8, 8)]:
            x = matrix(gen, rows, cols, xd, pad, offset, mean=0.3)
            weight = matrix(gen, 1, cols, xd, offset=offset, mean=1.0, sigma=0.2)[0]
            bias = matrix(gen, 1, cols, yd, sigma=0.2)[0]
            check_forward(x, weight, bias, EPS, yd, pad, offset, f"{rows}x{cols} {xd}->{yd}")


@pytest.mark.parametrize("rows", [1, 2, 15, 16, 17, 4097, 70001])
@pytest.mark.parametrize("cols", [40, 200, 512, 640])
def test_forward_rows(rows, cols):
    check_forward(matrix(generator(rows), rows, cols, BF), None, None, EPS, BF, 0, 0, f"{rows}x{cols}")


@pytest.mark.parametrize("weight,bias", itertools.product([True, False], repeat=2))
def test_forward_without_weight_or_bias(weight, bias):
    gen = generator(5)
    x = matrix(gen, 9, 300, F)
    check_forward(x, matrix(gen, 1, 300, F)[0] if weight else None, matrix(gen, 1, 300, BF)[0] if bias else None,
                  EPS, F, 0, 0, "optional")


def test_forward_mean_large_against_spread():
    """Values near 4096 with a spread of 1/16: a sum of squares minus the square
    of the mean would have nothing left."""
    gen = generator(6)
    check_forward(matrix(gen, 33, 1000, F, mean=4096.0, sigma=1 / 16), None, None, EPS, F, 0, 0, "large mean")


def test_forward_constant_and_nonfinite_rows():
    """Constant rows give the bias; a row with an infinity or a NaN is NaN
    throughout and leaves its neighbours, in the same wave or not, alone."""
    gen = generator(7)
    for cols in (100, 512, 1500):
        x = matrix(gen, 40, cols, F)
        bias = matrix(gen, 1, cols, F)[0]
        x[3] = 2.5
        x[5, cols // 2], x[8, 0], x[9, cols - 1] = float("inf"), float("-inf"), float("nan")
        y, rstd = Out(40, cols, F), Out(1, 40, F)
        T.taco_layer_norm(x, None, bias, EPS, y.t, rstd=rstd.vector())
        torch.cuda.synchronize()
        y.check("nonfinite")
        assert torch.equal(y.t[3], bias)
        bad = torch.tensor([5, 8, 9], device=DEV)
        assert bool(torch.isnan(y.t[bad]).all())
        good = [i for i in range(40) if i not in (3, 5, 8, 9)]
        clean = Out(len(good), cols, F)
        T.taco_layer_norm(x[good], None, bias, EPS, clean.t)
        torch.cuda.synchronize()
        assert torch.equal(y.t[good], clean.t)


def test_between_slices_of_one_tensor():
    """x and y are columns of one tensor, side by side; the rest of it stays."""
    gen = generator(17)
    rows, cols = 50, 136
    for dt in (BF, F):
        wide = matrix(gen, rows, 3 * cols, dt)
        before = wide.clone()
        T.taco_layer_norm(wide[:, cols:2 * cols], None, None, EPS, wide[:, :cols])
        want = torch.empty(rows, cols, dtype=dt, device=DEV)
        T.taco_layer_norm(before[:, cols:2 * cols].contiguous(), None, None, EPS, want)
        torch.cuda.synchronize()
        assert torch.equal(wide[:, :cols], want) and torch.equal(wide[:, cols:], before[:, cols:])
        with pytest.raises(T.TacoError):
            T.taco_layer_norm(wide[:, cols:2 * cols], None, None, EPS, wide[:, 2 * cols - 1:3 * cols - 1])


def backward64(dy, x, weight, mean, rstd):
    dy, x, mean, rstd = dy.double(), x.double(), mean.double()[:, None], rstd.double()[:, None]
    xhat = (x - mean) * rstd
    g = dy * (1.0 if weight is None else weight.double())
    a, b = g.mean(1, keepdim=True), (g * xhat).mean(1, keepdim=True)
    size = rstd * (g.abs() + g.abs().mean(1, keepdim=True) + xhat.abs() * (g * xhat).abs().mean(1, keepdim=True))
    return {"dx": ((g - a - xhat * b) * rstd, size), "dweight": ((dy * xhat).sum(0), (dy * xhat).abs().sum(0)),
            "dbias": (dy.sum(0), dy.abs().sum(0))}


def check_backward(gen, rows, cols, xd, dyd, dxd, pad, offset, what, weight=True, want=("dx", "dweight", "dbias"),
                   wd=F):
    x = matrix(gen, rows, cols, xd, pad, offset, mean=0.3)
    dy = matrix(gen, rows, cols, dyd, pad, offset)
    w = matrix(gen, 1, cols, xd, mean=1.0, sigma=0.2)[0] if weight else None
    mean = x.float().mean(1)
    rstd = (x.float().var(1, unbiased=False) + EPS).rsqrt()
    outs = {"dx": Out(rows, cols, dxd, pad, offset), "dweight": Out(1, cols, wd), "dbias": Out(1, cols, wd)}
    size = T.taco_layer_norm_backward_workspace_bytes(rows, cols)
    ws = Out(1, size // 4, F)
    T.taco_layer_norm_backward(dy, x, w, mean, rstd, dx=outs["dx"].t if "dx" in want else None,
                               dweight=outs["dweight"].vector() if "dweight" in want else None,
                               dbias=outs["dbias"].vector() if "dbias" in want else None,
                               workspace=ws.vector().view(torch.uint8))
    torch.cuda.synchronize()
    guard = torch.cat([ws.bits[:ws.lo], ws.bits[ws.hi:]])
    assert bool((guard == ws.mark).all()), f"{what}: wrote outside the workspace"
    refs = backward64(dy, x, w, mean, rstd)
    adds = -(-rows // 512) + 160 + 8
    for n in want:
        outs[n].check(f"{what} {n}")
        ref, size = refs[n]
        moved = (128 if n == "dx" else adds + 8) * U32 * size
        got = outs[n].t if n == "dx" else outs[n].vector()
        within(got, ref, moved + UNIT[got.dtype] * (ref.abs() + moved), f"{what} {n}")


@pytest.mark.parametrize("cols", WIDTHS)
def test_backward_widths(cols):
    for n, (xd, dyd, dxd) in enumerate([(BF, BF, BF), (F, BF, BF), (F, F, F), (BF, F, BF)]):
        gen = generator(cols * 10 + n)
        for rows, pad, offset in [(1, 0, 0), (3, 3, 1), (37, 8, 8)]:
            check_backward(gen, rows, cols, xd, dyd, dxd, pad, offset, f"{rows}x{cols} {xd},{dyd}->{dxd}")


@pytest.mark.parametrize("rows", [2, 16, 17, 511, 512, 513, 9001])
@pytest.mark.parametrize("cols", [40, 200, 512, 640])
def test_backward_rows(rows, cols):
    check_backward(generator(rows), rows, cols, BF, BF, BF, 0, 0, f"{rows}x{cols}")


@pytest.mark.parametrize("want", [("dx",), ("dweight",), ("dbias",), ("dx", "dbias"), ("dweight", "dbias")])
def test_backward_parts(want):
    for weight in (True, False):
        check_backward(generator(8), 70, 333, BF, BF, F, 0, 0, f"{want}", weight=weight, want=want, wd=BF)


def test_backward_of_no_rows_clears_the_sums():
    x = torch.empty(0, 50, dtype=F, device=DEV)
    none = torch.empty(0, dtype=F, device=DEV)
    dw, db = Out(1, 50, F), Out(1, 50, BF)
    T.taco_layer_norm_backward(x, x, None, none, none, dx=torch.empty_like(x), dweight=dw.vector(), dbias=db.vector())
    T.taco_layer_norm(x, None, None, EPS, torch.empty_like(x))
    torch.cuda.synchronize()
    dw.check("dweight")
    db.check("dbias")
    assert not dw.vector().any() and not db.vector().any()


def test_backward_against_differences():
    """Directional derivatives of sum(y * c), y from the definition in float64,
    by central differences of step 1e-4: their error is below 1e-7 of the
    derivative's terms, far below the float32 gradients' tolerance."""
    gen = generator(9)
    rows, cols, h = 12, 200, 1e-4
    x, dy = matrix(gen, rows, cols, F, mean=0.3), matrix(gen, rows, cols, F)
    w, b = matrix(gen, 1, cols, F, mean=1.0, sigma=0.2)[0], matrix(gen, 1, cols, F)[0]
    mean, rstd = torch.empty(rows, device=DEV), torch.empty(rows, device=DEV)
    y = torch.empty_like(x)
    T.taco_layer_norm(x, w, b, EPS, y, mean=mean, rstd=rstd)
    dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty_like(b)
    ws = torch.empty(T.taco_layer_norm_backward_workspace_bytes(rows, cols), dtype=torch.uint8, device=DEV)
    T.taco_layer_norm_backward(dy, x, w, mean, rstd, dx=dx, dweight=dw, dbias=db, workspace=ws)

    def loss(x_, w_, b_):
        return float((forward64(x_, w_, b_, EPS)[0] * dy.double()).sum())

    for seed in range(3):
        g = generator(100 + seed)
        vx = torch.randn(rows, cols, generator=g, device=DEV).double()
        vw, vb = torch.randn(cols, generator=g, device=DEV).double(), torch.randn(cols, generator=g, device=DEV).double()
        X, Wt, B = x.double(), w.double(), b.double()
        for got, vec, plus, minus in [
                (dx, vx, loss(X + h * vx, Wt, B), loss(X - h * vx, Wt, B)),
                (dw, vw, loss(X, Wt + h * vw, B), loss(X, Wt - h * vw, B)),
                (db, vb, loss(X, Wt, B + h * vb), loss(X, Wt, B - h * vb))]:
            terms = (got.double() * vec).abs().sum()
            diff = (plus - minus) / (2 * h)
            assert abs(float((got.double() * vec).sum()) - diff) <= 1e-5 * float(terms)


def test_on_another_stream_and_in_a_graph():
    """Calls on a side stream, and captured once and replayed on new inputs,
    give what eager calls on the current stream give, bit for bit."""
    gen = generator(10)
    rows, cols = 100, 1000
    xs = [matrix(gen, rows, cols, BF) for _ in range(3)]
    dys = [matrix(gen, rows, cols, BF) for _ in range(3)]
    w = matrix(gen, 1, cols, F)[0]
    size = T.taco_layer_norm_backward_workspace_bytes(rows, cols)

    def buffers():
        return dict(y=torch.zeros(rows, cols, dtype=BF, device=DEV), mean=torch.zeros(rows, device=DEV),
                    rstd=torch.zeros(rows, device=DEV), dx=torch.zeros(rows, cols, dtype=BF, device=DEV),
                    dw=torch.zeros(cols, device=DEV), ws=torch.zeros(size, dtype=torch.uint8, device=DEV))

    def step(x, dy, o, stream=None):
        T.taco_layer_norm(x, w, None, EPS, o["y"], mean=o["mean"], rstd=o["rstd"], stream=stream)
        T.taco_layer_norm_backward(dy, x, w, o["mean"], o["rstd"], dx=o["dx"], dweight=o["dw"], workspace=o["ws"],
                                   stream=stream)

    eager = []
    for x, dy in zip(xs, dys):
        o = buffers()
        step(x, dy, o)
        torch.cuda.synchronize()
        eager.append(o)
    side = torch.cuda.Stream()
    o = buffers()
    torch.cuda.synchronize()
    step(xs[0], dys[0], o, stream=side)
    side.synchronize()
    for n in ("y", "mean", "rstd", "dx", "dw"):
        assert torch.equal(o[n], eager[0][n]), n
    x, dy, o = xs[0].clone(), dys[0].clone(), buffers()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step(x, dy, o, stream=side)
    for i in (1, 0, 2):
        x.copy_(xs[i])
        dy.copy_(dys[i])
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for n in ("y", "mean", "rstd", "dx", "dw"):
            assert torch.equal(o[n], eager[i][n]), (i, n)
