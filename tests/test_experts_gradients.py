"""The gradients of the products by group in large tiles, and asked for one by
one: exactly in whole numbers, and within the tolerances of test_experts.py in
real ones. test_experts_launches.py holds these sizes and those of test_experts.py
to the kernels that they are there for."""

import itertools

import pytest
import torch

import quantized_compression_tensor_amd as T
from tests import test_experts as E
from tests.layers_util import Out, generator
from tests.test_experts import Case, Rows, cid, poison, three, whole, whole3
from tests.test_layers_linear import F, NONE, RELU, act64, slope64, space

pytestmark = pytest.mark.gpu

# large tiles of dx and of dw (also of 65 groups, and with empty ones), or of one of them, with edges inside the
# tiles, in place and packed. (N, of a plain projection; a gated one has as many weight rows with half of it.)
LARGE = [Case(3, 6500, 2056, 2056), Case(3, 6400, 2050, 2051, "some", 2, 5, 1, 1), Case(6, 6600, 1112, 2056, "some", 1, 0),
         Case(1, 7000, 3080, 4088, "one", 0, 3), Case(3, 4300, 1556, 3085, "even", 5, 1, 3), Case(65, 17000, 522, 200),
         Case(65, 16900, 520, 201, "even", 0, 2, 1), Case(2, 6200, 264, 2056), Case(2, 600, 5120, 1032, "even")]
# each height of dx's tiles, in place and not, with K whole and cut
ONE_BY_ONE = [Case(1, 2, 24, 12, pad=1), Case(8, 100, 136, 264), Case(5, 90, 130, 265, "some", 1, 2, 1, 1),
              Case(4, 200, 136, 264, "some", 0, 3), Case(4, 190, 138, 263, "some", 2, 0, 0, 1), Case(3, 700, 264, 328),
              Case(3, 650, 266, 329, "some", 1, 1, 3), Case(3, 60, 4104, 72), Case(3, 170, 4104, 72, "some", 1),
              Case(2, 300, 4104, 136), Case(2, 300, 4102, 131, pad=1), Case(40, 300, 2060, 1544, "some", 3, 2),
              Case(2, 33, 24, 5)] + LARGE


def half(c):
    """The gated case with as many weight rows."""
    h = Case.__new__(Case)
    h.__dict__.update(c.__dict__, N=c.N // 2, name="gated-" + c.name)
    return h


@pytest.mark.parametrize("c", LARGE, ids=cid)
def test_large_exact(c):
    E.test_linear_backward_exact(c)
    E.test_gated_backward_exact(half(c))


@pytest.mark.parametrize("c", LARGE[:3] + LARGE[6:8], ids=cid)
def test_large_real(c):
    E.test_backward_real(half(c), E.SILU)


def subsets(names):
    return [s for n in range(1, len(names) + 1) for s in itertools.combinations(names, n)]


@pytest.mark.parametrize("c", ONE_BY_ONE, ids=cid)
def test_linear_one_by_one(c):
    """Every subset of the gradients, each where its array is given; the same call gives the same bits."""
    gen = generator(c.M + c.N + c.K)
    x, w = whole(gen, c.M, c.K, 3, c.pad, c.offset), whole3(gen, c.G, c.N, c.K, 3, c.pad, c.offset)
    d, z = whole(gen, c.M, c.N, 3, c.pad, c.offset), whole(gen, c.M, c.N, 2, c.pad, c.offset)
    poison(c, x, d, z)
    ws = space(T.taco_grouped_linear_backward_workspace_bytes(c.G, c.M, c.N, c.K))
    for act in (NONE, RELU):
        want = {k: [] for k in ("dx", "dw", "dbias")}
        for g, r in c.ranges():
            dz = d[r].double() * slope64(z[r].double(), act)
            want["dx"].append(dz @ w[g].double())
            want["dw"].append(dz.t() @ x[r].double())
            want["dbias"].append(dz.sum(0)[None])
        want = {k: torch.cat(v) for k, v in want.items()}
        for names in subsets(("dx", "dw", "dbias")):
            outs = {"dx": Rows(c.M, c.K, F, c.pad, c.offset), "dw": Out(c.G * c.N, c.K, F, c.pad, c.offset),
                    "dbias": Out(c.G, c.N, F, c.pad)}
            views = {k: three(outs[k].t, c.G) if k == "dw" else outs[k].t for k in names}
            T.taco_grouped_linear_backward(d, x, w, c.offsets(), act=act, preact=z if act else None, workspace=ws, **views)
            torch.cuda.synchronize()
            for k in names:
                got = outs[k].t
                if k == "dx":
                    outs[k].check_rows(c.inside(), k)
                    got = got[c.inside()]
                else:
                    outs[k].check(k)
                assert torch.equal(got.double(), want[k]), (act, names, k)


@pytest.mark.parametrize("c", ONE_BY_ONE, ids=cid)
def test_gated_one_by_one(c):
    c = half(c)
    gen = generator(c.M + c.N + c.K)
    x, w = whole(gen, c.M, c.K, 2, c.pad, c.offset), whole3(gen, c.G, 2 * c.N, c.K, 2, c.pad, c.offset)
    d, z = whole(gen, c.M, c.N, 2, c.pad, c.offset), whole(gen, c.M, 2 * c.N, 2, c.pad, c.offset, F)
    poison(c, x, d, z)
    ws = space(T.taco_grouped_gated_linear_backward_workspace_bytes(c.G, c.M, c.N, c.K))
    want = {"dx": [], "dw": []}
    for g, r in c.ranges():
        d64, a, u = d[r].double(), z[r, :c.N].double(), z[r, c.N:].double()
        dz = torch.cat([d64 * u * slope64(a, RELU), d64 * act64(a, RELU)], 1)
        want["dx"].append(dz @ w[g].double())
        want["dw"].append(dz.t() @ x[r].double())
    want = {k: torch.cat(v) for k, v in want.items()}
    for names in subsets(("dx", "dw")):
        outs = {"dx": Rows(c.M, c.K, F, c.pad, c.offset), "dw": Out(c.G * 2 * c.N, c.K, F, c.pad, c.offset)}
        views = {k: three(outs[k].t, c.G) if k == "dw" else outs[k].t for k in names}
        T.taco_grouped_gated_linear_backward(d, x, w, c.offsets(), act=RELU, preact=z, workspace=ws, **views)
        torch.cuda.synchronize()
        for k in names:
            got = outs[k].t
            if k == "dx":
                outs[k].check_rows(c.inside(), k)
                got = got[c.inside()]
            else:
                outs[k].check(k)
            assert torch.equal(got.double(), want[k]), (names, k)


@pytest.mark.parametrize("c", [LARGE[1], LARGE[6], Case(32, 2000, 520, 1000, "some", 0, 48), Case(3, 170, 4104, 72, "some", 1)],
                         ids=cid)
def test_the_same_call_gives_the_same_bits(c):
    """Real values, a workspace of other contents, and other work between the calls."""
    gen = generator(c.M)
    x, d, z = (E.matrix(gen, c.M, n, E.BF, c.pad, c.offset) for n in (c.K, c.N, c.N))
    w = E.matrix(gen, c.G * c.N, c.K, E.BF, sigma=0.1).view(c.G, c.N, c.K)
    size, results = T.taco_grouped_linear_backward_workspace_bytes(c.G, c.M, c.N, c.K), []
    for fill in (0, 255):
        dx, dw, db = torch.zeros(c.M, c.K, dtype=E.BF, device=E.DEV), torch.empty_like(w), torch.empty(c.G, c.N, device=E.DEV)
        T.taco_grouped_linear_backward(d, x, w, c.offsets(), act=E.GELU, preact=z, dx=dx, dw=dw, dbias=db,
                                       workspace=torch.full((size,), fill, dtype=torch.uint8, device=E.DEV))
        results.append((dx, dw, db))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(*results))
