"""The projections by group, plain and gated, forward and backward, against
their formulas in float64: exactly in whole numbers, and within the tolerances
of test_layers_linear.py in real ones. Rows of no group must keep what they
held."""

import math

import pytest
import torch

import quantized_compression_tensor_amd as T
from tests.layers_util import DEV, U32, UNIT, Out, generator, matrix, within
from tests.test_layers_linear import ACTS, BF, F, GELU, NONE, RELU, SILU, act64, product64, slope64, space

pytestmark = pytest.mark.gpu


def sizes_of(rows, groups, how):
    """Rows of each group, `rows` in all."""
    g = torch.Generator()
    g.manual_seed(rows + groups)
    if how == "one":
        s = [0] * groups
        s[groups * 2 // 3] = rows
    elif how == "even":
        s = [rows // groups + (i < rows % groups) for i in range(groups)]
    else:                          # some groups empty, some far larger
        like = torch.randn(groups, generator=g).exp() * (torch.rand(groups, generator=g) < 0.7)
        like[groups - 1] += 0.01
        s = torch.bincount(torch.multinomial(like, rows, True, generator=g), minlength=groups).tolist() if rows else [0] * groups
    assert sum(s) == rows
    return s


class Case:
    """groups, rows of them, N, K, distribution, rows before and after, pad, offset."""

    def __init__(self, groups, rows, N, K, how="some", before=0, after=0, pad=0, offset=0):
        self.G, self.N, self.K, self.pad, self.offset = groups, N, K, pad, offset
        self.M = before + rows + after
        sizes = sizes_of(rows, groups, how)
        self.name = f"{groups}g-{rows}x{N}x{K}-{how}-b{before}a{after}p{pad}o{offset}"
        o = [before]
        for s in sizes:
            o.append(o[-1] + s)
        self.o = o

    def offsets(self):
        return torch.tensor(self.o, dtype=torch.int32, device=DEV)

    def ranges(self):
        return [(g, slice(self.o[g], self.o[g + 1])) for g in range(self.G)]

    def inside(self):
        m = torch.zeros(self.M, dtype=torch.bool, device=DEV)
        m[self.o[0]:self.o[-1]] = True
        return m


CASES = [
    Case(1, 1, 1, 1), Case(3, 2, 7, 9, pad=1, offset=1), Case(64, 8, 96, 128, "even"), Case(8, 1, 40, 264),
    Case(4, 30, 33, 65, pad=3, offset=1), Case(5, 27, 130, 72, "one", 2, 3), Case(1000, 31, 24, 40),
    Case(2, 33, 128, 128, "one"), Case(12, 100, 300, 328, "some", 5, 7, 8, 8), Case(70, 300, 72, 136, "some", 0, 9),
    Case(300, 2000, 40, 72), Case(1024, 1500, 16, 24, "some", 3, 0), Case(8, 400, 136, 64, "even"),
    Case(6, 333, 257, 193, "some", 1, 60, 3, 1), Case(4, 900, 264, 328, "some", 0, 31), Case(3, 1000, 515, 200, "one"),
    Case(7, 3500, 264, 136), Case(2, 700, 1032, 1288, "some", 11, 5), Case(4, 6000, 520, 72, "some", 8, 8, 24, 16),
    Case(8, 8200, 1536, 72, "even"), Case(3, 9000, 1540, 136, "some", 4, 100), Case(9, 0, 24, 40, "even", 6, 7),
    Case(5, 4097, 1100, 80, "one", 1, 2, 5, 3),
    # many tiles of dw with short sums; few tiles with a long K, forward and dx; 64 and 65 groups
    Case(40, 300, 2060, 1544, "some", 3, 2), Case(3, 70, 136, 4104, "some"), Case(2, 100, 4100, 136, "some", 1, 0, 1),
    # K cut, in tiles of 64 and 128 rows, in place and not: forward, and dx
    Case(2, 100, 136, 4104, "some"), Case(2, 300, 200, 4104, "some", 1, 1), Case(2, 90, 130, 4099, "some", 0, 2, 1, 1),
    Case(2, 300, 200, 4101, "some", 0, 0, 1, 1), Case(2, 300, 4104, 136), Case(3, 60, 4104, 72), Case(2, 300, 4101, 130, pad=1),
    # ranges of more than eight rows in dbias
    Case(3, 40000, 24, 16, "some", 2, 9), Case(300, 36000, 17, 8),
    Case(64, 3000, 136, 72), Case(65, 3000, 136, 72, "some", 1, 1), Case(3, 1600, 1000, 1001, "some", 0, 0, 2, 1),
    # 32 to 64 rows to a group and many tiles, in place and not; up to 32 rows times many weights
    Case(20, 1000, 1800, 136, "some", 2, 3), Case(20, 900, 1800, 137, "even", 1, 0, 1, 1),
    Case(9, 32, 1540, 1544, "some", 1, 2), Case(9, 30, 1541, 1543, "some", 0, 1, 2, 1), Case(32, 32, 1540, 1544, "even"),
]


def cid(c):
    return c.name


def whole3(gen, groups, rows, cols, most, pad=0, offset=0, dtype=BF):
    """Whole numbers in a [groups, rows, cols] view with its rows cols + pad apart; NaN between them."""
    m = matrix(gen, groups * rows, cols, dtype, pad, offset)
    m.copy_(torch.randint(-most, most + 1, m.shape, generator=gen, device=DEV))
    return torch.as_strided(m, (groups, rows, cols), (rows * (cols + pad), cols + pad, 1), m.storage_offset())


def whole(gen, rows, cols, most, pad=0, offset=0, dtype=BF):
    return whole3(gen, 1, rows, cols, most, pad, offset, dtype)[0]


class Rows(Out):
    """An output of which only some rows are written."""

    def check_rows(self, inside, what):
        rows, wide = self.t.shape[0], (self.hi - self.lo) // max(1, self.t.shape[0])
        want = torch.zeros_like(self.bits, dtype=torch.bool)
        want[self.lo:self.hi].view(rows, wide)[:, :self.cols] = inside[:, None]
        marked = self.bits == self.mark
        assert bool(marked[~want].all()), f"{what}: wrote outside the groups' rows"
        assert not bool(marked[want].any()), f"{what}: left elements unwritten"


def three(t, groups):
    """An output matrix [groups * rows, cols] as the binding takes it."""
    rows = t.shape[0] // groups
    return torch.as_strided(t, (groups, rows, t.shape[1]), (rows * t.stride(0), t.stride(0), 1), t.storage_offset())


def products(c, x, w, bias=None):
    """z in float64, zeros in rows of no group."""
    z = torch.zeros(c.M, w.shape[1], dtype=torch.float64, device=DEV)
    for g, r in c.ranges():
        z[r] = x[r].double() @ w[g].double().t()
        if bias is not None:
            z[r] += bias[g].double()
    return z


def poison(c, *tensors):
    """NaN in the rows of no group: nothing may come from there."""
    for t in tensors:
        t[~c.inside()] = math.nan


# ---------------------------------------------------------------- exactly --

@pytest.mark.parametrize("c", CASES, ids=cid)
def test_linear_exact(c):
    gen = generator(c.M + c.N + c.K)
    x, w = whole(gen, c.M, c.K, 3, c.pad, c.offset), whole3(gen, c.G, c.N, c.K, 3, c.pad, c.offset)
    b = whole(gen, c.G, c.N, 8, c.pad, c.offset)
    poison(c, x)
    out, z = Rows(c.M, c.N, F, c.pad, c.offset), Rows(c.M, c.N, F, c.pad, c.offset)
    ws = space(T.taco_grouped_linear_workspace_bytes(c.G, c.M, c.N, c.K))
    T.taco_grouped_linear(x, w, c.offsets(), out.t, bias=b, act=RELU, preact=z.t, workspace=ws)
    plain = Rows(c.M, c.N, BF, c.pad, c.offset)
    T.taco_grouped_linear(x, w, c.offsets(), plain.t, workspace=ws)
    torch.cuda.synchronize()
    inside = c.inside()
    for o, n in ((out, "out"), (z, "preact"), (plain, "plain")):
        o.check_rows(inside, n)
    want = products(c, x, w, b)[inside]
    assert torch.equal(z.t[inside].double(), want)
    assert torch.equal(out.t[inside].double(), want.clamp(min=0))
    assert torch.equal(plain.t[inside], products(c, x, w)[inside].to(BF))


@pytest.mark.parametrize("c", CASES, ids=cid)
def test_gated_exact(c):
    gen = generator(c.M + c.N + c.K)
    x, w = whole(gen, c.M, c.K, 1, c.pad, c.offset), whole3(gen, c.G, 2 * c.N, c.K, 1, c.pad, c.offset)
    poison(c, x)
    out, z = Rows(c.M, c.N, F, c.pad, c.offset), Rows(c.M, 2 * c.N, F, c.pad, c.offset)
    T.taco_grouped_gated_linear(x, w, c.offsets(), out.t, act=RELU, preact=z.t,
                                workspace=space(T.taco_grouped_gated_linear_workspace_bytes(c.G, c.M, c.N, c.K)))
    torch.cuda.synchronize()
    inside = c.inside()
    out.check_rows(inside, "out")
    z.check_rows(inside, "preact")
    want = products(c, x, w)[inside]
    assert torch.equal(z.t[inside].double(), want)
    assert torch.equal(out.t[inside].double(), want[:, :c.N].clamp(min=0) * want[:, c.N:])


@pytest.mark.parametrize("c", CASES, ids=cid)
def test_linear_backward_exact(c):
    gen = generator(c.M + c.N + c.K)
    x, w = whole(gen, c.M, c.K, 3, c.pad, c.offset), whole3(gen, c.G, c.N, c.K, 3, c.pad, c.offset)
    d, z = whole(gen, c.M, c.N, 3, c.pad, c.offset), whole(gen, c.M, c.N, 2, c.pad, c.offset)
    poison(c, x, d, z)
    inside = c.inside()
    for act in (NONE, RELU):
        dx, dw = Rows(c.M, c.K, F, c.pad, c.offset), Out(c.G * c.N, c.K, F, c.pad, c.offset)
        db = Out(c.G, c.N, F, c.pad)
        T.taco_grouped_linear_backward(d, x, w, c.offsets(), act=act, preact=z if act else None, dx=dx.t,
                                       dw=three(dw.t, c.G), dbias=db.t,
                                       workspace=space(T.taco_grouped_linear_backward_workspace_bytes(c.G, c.M, c.N, c.K)))
        torch.cuda.synchronize()
        dx.check_rows(inside, "dx")
        dw.check("dw")
        db.check("dbias")
        for g, r in c.ranges():
            dz = d[r].double() * slope64(z[r].double(), act)
            assert torch.equal(dx.t[r].double(), dz @ w[g].double()), (act, g)
            assert torch.equal(three(dw.t, c.G)[g].double(), dz.t() @ x[r].double()), (act, g)
            assert torch.equal(db.t[g].double(), dz.sum(0)), (act, g)


@pytest.mark.parametrize("c", CASES, ids=cid)
def test_gated_backward_exact(c):
    gen = generator(c.M + c.N + c.K)
    x, w = whole(gen, c.M, c.K, 2, c.pad, c.offset), whole3(gen, c.G, 2 * c.N, c.K, 2, c.pad, c.offset)
    d, z = whole(gen, c.M, c.N, 2, c.pad, c.offset), whole(gen, c.M, 2 * c.N, 2, c.pad, c.offset, F)
    poison(c, x, d, z)
    dx, dw = Rows(c.M, c.K, F, c.pad, c.offset), Out(c.G * 2 * c.N, c.K, BF, c.pad, c.offset)
    T.taco_grouped_gated_linear_backward(
        d, x, w, c.offsets(), act=RELU, preact=z, dx=dx.t, dw=three(dw.t, c.G),
        workspace=space(T.taco_grouped_gated_linear_backward_workspace_bytes(c.G, c.M, c.N, c.K)))
    torch.cuda.synchronize()
    dx.check_rows(c.inside(), "dx")
    dw.check("dw")
    for g, r in c.ranges():
        d64, a, u = d[r].double(), z[r, :c.N].double(), z[r, c.N:].double()
        dz = torch.cat([d64 * u * slope64(a, RELU), d64 * act64(a, RELU)], 1)
        assert torch.equal(dx.t[r].double(), dz @ w[g].double())
        assert torch.equal(three(dw.t, c.G)[g], (dz.t() @ x[r].double()).to(BF))


# ------------------------------------------------------------ real values --

REAL = [Case(6, 20, 136, 520, "some", 1, 2), Case(5, 90, 264, 333, "some", 0, 4, 1), Case(3, 200, 520, 264),
        Case(4, 700, 264, 520, "some", 9, 0), Case(2, 1500, 1032, 264, "even")]


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("c", REAL, ids=cid)
def test_forward_real(c, act):
    gen = generator(c.M + c.N + act)
    x = matrix(gen, c.M, c.K, BF, c.pad, c.offset)
    w = matrix(gen, c.G * 2 * c.N, c.K, BF, sigma=3 / math.sqrt(c.K)).view(c.G, 2 * c.N, c.K)
    b = matrix(gen, c.G, c.N, F)
    inside, half = c.inside(), w[:, :c.N].contiguous()
    for od, zd in ((BF, F), (F, BF)):
        out, zo = Rows(c.M, c.N, od, c.pad), Rows(c.M, c.N, zd)
        T.taco_grouped_linear(x, half, c.offsets(), out.t, bias=b, act=act, preact=zo.t,
                              workspace=space(T.taco_grouped_linear_workspace_bytes(c.G, c.M, c.N, c.K)))
        gout, gz = Rows(c.M, c.N, od, c.pad), Rows(c.M, 2 * c.N, zd)
        T.taco_grouped_gated_linear(x, w, c.offsets(), gout.t, act=act, preact=gz.t,
                                    workspace=space(T.taco_grouped_gated_linear_workspace_bytes(c.G, c.M, c.N, c.K)))
        torch.cuda.synchronize()
        for o in (out, zo, gout, gz):
            o.check_rows(inside, "output")
        for g, r in c.ranges():
            z, size = product64(x[r], half[g])
            z, size = z + b[g].double(), size + b[g].double().abs()
            tz = (c.K / 4 + 64) * U32 * size
            within(zo.t[r], z, tz + UNIT[zd] * (z.abs() + tz), "preact")
            want = act64(z, act)
            t = 1.13 * tz + 32 * U32 * z.abs() + U32 * want.abs()
            within(out.t[r], want, t + UNIT[od] * (want.abs() + t), "out")
            z, size = product64(x[r], w[g])
            tz = (c.K / 4 + 64) * U32 * size
            within(gz.t[r], z, tz + UNIT[zd] * (z.abs() + tz), "gated preact")
            v, u = act64(z[:, :c.N], act), z[:, c.N:]
            tv = 1.13 * tz[:, :c.N] + 32 * U32 * z[:, :c.N].abs()
            t = tv * u.abs() + v.abs() * tz[:, c.N:] + tv * tz[:, c.N:] + U32 * (v * u).abs()
            within(gout.t[r], v * u, t + UNIT[od] * ((v * u).abs() + t), "gated out")


def check_group(dz, tdz, x, w, dx, dw):
    """One group's gradients from its dz, of which the kernel's operand is tdz off."""
    for got, a, ta, b, n, what in ((dx, dz, tdz, w.t(), w.shape[0], "dx"), (dw, dz.t(), tdz.t(), x.t(), x.shape[0], "dw")):
        want, size = product64(a, b)
        off = ta @ b.double().abs().t()
        t = off + (n / 4 + 64) * U32 * (size + off)
        within(got, want, t + UNIT[got.dtype] * (want.abs() + t), what)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("c", REAL, ids=cid)
def test_backward_real(c, act):
    gen = generator(c.M + c.N + act)
    x = matrix(gen, c.M, c.K, BF, c.pad, c.offset)
    w = matrix(gen, c.G * 2 * c.N, c.K, BF, sigma=0.1).view(c.G, 2 * c.N, c.K)
    half = w[:, :c.N].contiguous()
    inside = c.inside()
    for zd, gd in ((BF, BF), (F, F)):
        d, z = matrix(gen, c.M, c.N, BF, c.pad), matrix(gen, c.M, 2 * c.N, zd, c.pad, sigma=2.0)
        dx, dw, db = Rows(c.M, c.K, gd, c.pad), Out(c.G * c.N, c.K, gd), Out(c.G, c.N, F)
        T.taco_grouped_linear_backward(d, x, half, c.offsets(), act=act, preact=z[:, :c.N], dx=dx.t,
                                       dw=three(dw.t, c.G), dbias=db.t,
                                       workspace=space(T.taco_grouped_linear_backward_workspace_bytes(c.G, c.M, c.N, c.K)))
        gx, gw = Rows(c.M, c.K, gd, c.pad), Out(c.G * 2 * c.N, c.K, gd)
        T.taco_grouped_gated_linear_backward(
            d, x, w, c.offsets(), act=act, preact=z, dx=gx.t, dw=three(gw.t, c.G),
            workspace=space(T.taco_grouped_gated_linear_backward_workspace_bytes(c.G, c.M, c.N, c.K)))
        torch.cuda.synchronize()
        for o in (dx, gx):
            o.check_rows(inside, "dx")
        for o in (dw, db, gw):
            o.check("gradient")
        for g, r in c.ranges():
            d64, a, u = d[r].double(), z[r, :c.N].double(), z[r, c.N:].double()
            dz = d64 * slope64(a, act)
            t32 = torch.zeros_like(dz) if act == NONE else 64 * U32 * d64.abs()
            check_group(dz, t32 + (0 if act == NONE else 2.0 ** -8) * (dz.abs() + t32), x[r], half[g], dx.t[r],
                        three(dw.t, c.G)[g])
            rows = r.stop - r.start
            within(db.t[g], dz.sum(0), t32.sum(0) + (rows / 4 + 64) * U32 * (dz.abs() + t32).sum(0)
                   + U32 * dz.sum(0).abs(), "dbias")
            dz = torch.cat([d64 * u * slope64(a, act), d64 * act64(a, act)], 1)
            t32 = torch.cat([66 * U32 * (d64 * u).abs(), 34 * U32 * (d64 * a).abs()], 1)
            check_group(dz, t32 + 2.0 ** -8 * (dz.abs() + t32), x[r], w[g], gx.t[r], three(gw.t, c.G)[g])


def test_gradients_against_differences():
    """The gradients of sum(out * t) against central differences of the forward
    pass: gelu's third derivative is below 1.2 in magnitude, so a step of h in
    direction v of z is off by 0.2 h^2 |v|^3 in each element; and the outputs' own
    errors, (K / 4 + 96) U32 of the sums of magnitudes, divided by h."""
    gen = generator(77)
    c = Case(3, 40, 24, 32, "some", 1, 1)
    x, w = matrix(gen, c.M, c.K, BF), matrix(gen, c.G * c.N, c.K, BF, sigma=0.2).view(c.G, c.N, c.K)
    b, t = matrix(gen, c.G, c.N, F), matrix(gen, c.M, c.N, BF)
    inside = c.inside()
    ws = space(T.taco_grouped_linear_workspace_bytes(c.G, c.M, c.N, c.K))

    def loss(bias):
        out = torch.zeros(c.M, c.N, device=DEV)
        T.taco_grouped_linear(x, w, c.offsets(), out, bias=bias, act=GELU, workspace=ws)
        return (out[inside].double() * t[inside].double())

    z = torch.empty(c.M, c.N, device=DEV)
    T.taco_grouped_linear(x, w, c.offsets(), torch.empty(c.M, c.N, device=DEV), bias=b, act=GELU, preact=z, workspace=ws)
    db = torch.empty(c.G, c.N, device=DEV)
    T.taco_grouped_linear_backward(t, x, w, c.offsets(), act=GELU, preact=z, dbias=db,
                                   workspace=space(T.taco_grouped_linear_backward_workspace_bytes(c.G, c.M, c.N, c.K)))
    h = 2.0 ** -6
    sizes = torch.zeros(c.M, c.N, dtype=torch.float64, device=DEV)
    for g, r in c.ranges():
        sizes[r] = product64(x[r], w[g])[1] + b[g].double().abs() + 1
    for g in range(c.G):
        step = torch.zeros_like(b)
        step[g] = h
        diff = (loss(b + step) - loss(b - step)) / (2 * h)
        per_column = torch.zeros(c.M, c.N, dtype=torch.float64, device=DEV)
        per_column[inside] = diff
        r = slice(c.o[g], c.o[g + 1])
        off = (0.2 * h * h + (c.K / 4 + 96) * U32 * sizes[r] / h) * t[r].double().abs()
        slope = (c.M / 4 + 64) * U32 * 1.13 * t[r].double().abs().sum(0)
        within(per_column[r].sum(0), db[g].double(), off.sum(0) + slope, f"dbias of group {g}")
        outside = torch.ones(c.M, dtype=torch.bool, device=DEV)
        outside[r] = False
        assert not bool(per_column[outside].any())      # no other group's


# ----------------------------------------------------------------- the rest --

def test_offsets_out_of_range_or_decreasing():
    """Values are unspecified where the offsets are no offsets, and nothing is
    written outside of the arrays; in range and not decreasing again, all is well."""
    gen = generator(9)
    G, M, N, K = 9, 500, 136, 72
    x, w = whole(gen, M, K, 2), whole3(gen, G, N, K, 2)
    d = whole(gen, M, N, 2)
    for o in ([0, 50, 40, 30, 400, 100, 600, 500, -7, 500], [-2 ** 31, 2 ** 31 - 1] * 5, [500] * 10, [0] * 9 + [2 ** 31 - 1],
              [100, 0, 500, 0, 500, 0, 500, 0, 500, 0]):
        offsets = torch.tensor(o, dtype=torch.int32, device=DEV)
        out, dx, dw, db = Out(M, N, F), Out(M, K, F), Out(G * N, K, F), Out(G, N, F)
        T.taco_grouped_linear(x, w, offsets, out.t, workspace=space(T.taco_grouped_linear_workspace_bytes(G, M, N, K)))
        T.taco_grouped_linear_backward(d, x, w, offsets, dx=dx.t, dw=three(dw.t, G), dbias=db.t,
                                       workspace=space(T.taco_grouped_linear_backward_workspace_bytes(G, M, N, K)))
        torch.cuda.synchronize()
        for t in (out, dx, dw, db):
            edge = torch.cat([t.bits[:t.lo], t.bits[t.hi:]])
            assert bool((edge == t.mark).all())
    # out of range, but not decreasing: the nearer end
    offsets = torch.tensor([-5, -1, 100, 100, 300, 499, 500, 501, 10 ** 9, 2 ** 31 - 1], dtype=torch.int32, device=DEV)
    out = Out(M, N, F)
    T.taco_grouped_linear(x, w, offsets, out.t, workspace=space(T.taco_grouped_linear_workspace_bytes(G, M, N, K)))
    torch.cuda.synchronize()
    out.check("out")
    o = offsets.clamp(0, M).tolist()
    for g in range(G):
        assert torch.equal(out.t[o[g]:o[g + 1]].double(), x[o[g]:o[g + 1]].double() @ w[g].double().t())


@pytest.mark.parametrize("rows,N,K", [(20, 40, 72), (100, 136, 200), (400, 264, 136), (900, 264, 130), (3000, 520, 264)])
def test_a_groups_nan_stays_in_it(rows, N, K):
    """Rows of NaN and infinities at the ends of one group leave the others' bits."""
    gen = generator(rows)
    G = 4
    o = [0, rows // 3, rows // 3 + rows // 4 + 1, rows // 2 + rows // 3, rows]
    offsets = torch.tensor(o, dtype=torch.int32, device=DEV)
    x, d, w = matrix(gen, rows, K, BF), matrix(gen, rows, N, BF), whole3(gen, G, N, K, 2)
    outs = []
    for bad in (False, True):
        if bad:
            x[o[1]], x[o[2] - 1], d[o[1]], d[o[2] - 1] = math.nan, math.inf, -math.inf, math.nan
        out, dx, dw, db = (torch.zeros(*s, device=DEV) for s in ((rows, N), (rows, K), (G, N, K), (G, N)))
        T.taco_grouped_linear(x, w, offsets, out, workspace=space(T.taco_grouped_linear_workspace_bytes(G, rows, N, K)))
        T.taco_grouped_linear_backward(d, x, w, offsets, dx=dx, dw=dw, dbias=db,
                                       workspace=space(T.taco_grouped_linear_backward_workspace_bytes(G, rows, N, K)))
        outs.append((out, dx, dw, db))
    torch.cuda.synchronize()
    live = torch.ones(rows, dtype=torch.bool, device=DEV)
    live[[o[1], o[2] - 1]] = False
    others = [0, 2, 3]
    for i, (was, now) in enumerate(zip(*outs)):
        part = live if i < 2 else others
        assert torch.equal(was[part], now[part]) and not bool(torch.isnan(now[part]).any())
        rest = now[~live] if i < 2 else now[1]
        assert not bool(torch.isfinite(rest).any()) if i != 1 else bool((~torch.isfinite(rest)).any())


def test_no_rows():
    w, o = torch.zeros(3, 24, 40, dtype=BF, device=DEV), torch.zeros(4, dtype=torch.int32, device=DEV)
    x, d = torch.empty(0, 40, dtype=BF, device=DEV), torch.empty(0, 24, dtype=BF, device=DEV)
    T.taco_grouped_linear(x, w, o, d)
    T.taco_grouped_gated_linear(x, w, o, d[:, :12])
    dw, db = torch.ones(3, 24, 40, device=DEV), torch.ones(3, 24, device=DEV)
    ws = space(T.taco_grouped_linear_backward_workspace_bytes(3, 0, 24, 40))
    T.taco_grouped_linear_backward(d, x, w, o, act=GELU, preact=d, dx=torch.empty_like(x), dw=dw, dbias=db, workspace=ws)
    torch.cuda.synchronize()
    assert not bool(dw.any()) and not bool(db.any())
    dw.fill_(1)
    T.taco_grouped_gated_linear_backward(torch.empty(0, 12, dtype=BF, device=DEV), x, w, o,
                                         preact=torch.empty(0, 24, device=DEV), dw=dw, workspace=ws)
    torch.cuda.synchronize()
    assert not bool(dw.any())


@pytest.mark.parametrize("rows", [5, 200, 1200])
def test_captured_with_other_offsets(rows):
    """A training step of a layer with experts on a stream of its own, captured
    and replayed with other rows and other groups, against the same step run
    eagerly."""
    gen = generator(rows)
    G, H, I, M = 6, 136, 264, rows + 40
    x, dy = matrix(gen, M, H, BF), matrix(gen, M, H, BF)
    w1 = matrix(gen, G * 2 * I, H, BF, sigma=0.1).view(G, 2 * I, H)
    w2, b2 = matrix(gen, G * H, I, BF, sigma=0.1).view(G, H, I), matrix(gen, G, H, BF)
    o = torch.zeros(G + 1, dtype=torch.int32, device=DEV)
    z, h, y = torch.zeros(M, 2 * I, dtype=BF, device=DEV), torch.zeros(M, I, dtype=BF, device=DEV), torch.zeros(M, H, dtype=BF, device=DEV)
    dh, dx = torch.zeros(M, I, dtype=BF, device=DEV), torch.zeros(M, H, dtype=BF, device=DEV)
    dw1, dw2, db2 = torch.zeros_like(w1), torch.zeros_like(w2), torch.zeros(G, H, device=DEV)
    size = max(T.taco_grouped_gated_linear_workspace_bytes(G, M, I, H), T.taco_grouped_linear_workspace_bytes(G, M, H, I),
               T.taco_grouped_gated_linear_backward_workspace_bytes(G, M, I, H),
               T.taco_grouped_linear_backward_workspace_bytes(G, M, H, I))
    ws = space(size)
    outs = (y, dx, dw1, dw2, db2)

    def step():
        T.taco_grouped_gated_linear(x, w1, o, h, preact=z, workspace=ws)
        T.taco_grouped_linear(h, w2, o, y, bias=b2, workspace=ws)
        T.taco_grouped_linear_backward(dy, h, w2, o, dx=dh, dw=dw2, dbias=db2, workspace=ws)
        T.taco_grouped_gated_linear_backward(dh, x, w1, o, preact=z, dx=dx, dw=dw1, workspace=ws)

    def set_groups(seed):
        s = sizes_of(rows + 5 * seed, G, "even" if seed % 2 else "some")
        o.copy_(torch.tensor([0] + s).cumsum(0).int() + seed)

    set_groups(0)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        step()
    stream.synchronize()
    eager = [t.clone() for t in outs]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for k in range(4):
        set_groups(k)
        if k:
            x.copy_(matrix(generator(k), M, H, BF))
        for t in (*outs, h, z, dh):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in outs]
        for t in (*outs, h, z, dh):
            t.zero_()
        step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, outs))
        if k == 0:
            assert all(torch.equal(a, b) for a, b in zip(got, eager))
