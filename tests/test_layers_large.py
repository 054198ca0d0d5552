"""The products' large tiles (256 x 256) over many steps of K, where every LDS
stage is filled again and read back, with K whole and cut and with edges inside
the tiles; exactly, in whole numbers, as in test_layers_linear.py. A test on
the CPU holds each size to the plan that it is here for."""

import os
import subprocess

import pytest
import torch

import quantized_compression_tensor_amd as T
from tests.conftest import ROOT
from tests.layers_util import Out, generator
from tests.test_layers_linear import BF, F, GELU, NONE, RELU, act64, slope64, whole

HIPCC = "/opt/rocm/bin/hipcc"

# (M, N, K, pad, cut): cut, whether K of the last round of tiles is cut. The
# rows of those without a pad can be loaded in place, the others are packed.
FORWARD = [(4100, 4104, 2056, 0, True), (4090, 4090, 1000, 0, False), (4099, 4101, 2057, 3, True)]
GATED = [(4100, 4104, 2056, 0, True), (4090, 2040, 1000, 0, False), (4099, 4101, 2057, 1, True)]
# (M, N, K, pad, dx, dw): of which product, True: large tiles with a cut K,
# False: without, None: small ones
BACKWARD = [(4100, 4104, 4112, 0, True, True), (4090, 1000, 4088, 0, False, None), (1000, 4088, 4088, 0, None, False),
            (2051, 4101, 8195, 5, True, True)]
GATED_BACKWARD = [(4100, 2056, 4104, 0, True, True), (4090, 504, 4088, 0, False, None),
                  (1000, 2044, 4088, 0, None, False), (4101, 2051, 4099, 1, True, True)]


def ids(s):
    return "x".join(map(str, s[:3])) + f"-p{s[3]}"


def plans(folder, lines):
    """What linear.hip's host code plans for each line."""
    if not os.path.exists(HIPCC):
        pytest.skip("hipcc not installed")
    import importlib.util
    spec = importlib.util.spec_from_file_location(
        "taco_build", os.path.join(ROOT, "quantized_compression_tensor_amd", "build.py"))
    build = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(build)
    exe = str(folder / "layers_plan")
    flags = [f for f in build.FLAGS if f != "-O3"]
    b = subprocess.run([HIPCC, *flags, "-O1", "-x", "hip", f"-I{build.CSRC}", os.path.join(ROOT, "tests", "layers_plan.cpp"),
                        "-o", exe], capture_output=True, text=True, timeout=600)
    assert b.returncode == 0, b.stderr[-3000:]
    r = subprocess.run([exe], input="\n".join(lines) + "\n", capture_output=True, text=True, timeout=60)
    assert r.returncode == 0
    return [[int(v) for v in line.split()] for line in r.stdout.splitlines()]


def test_sizes_take_the_plans_that_they_are_for(tmp_path):
    ask, expect = [], []
    for M, N, K, _, cut in FORWARD:
        ask.append(f"{M} {N} {K} linear"), expect.append(cut)
    for M, N, K, _, cut in GATED:
        ask.append(f"{M} {N} {K} gated"), expect.append(cut)
    for sizes, wide in ((BACKWARD, 1), (GATED_BACKWARD, 2)):
        for M, N, K, _, dx, dw in sizes:
            ask.append(f"{M} {K} {wide * N} linear"), expect.append(dx)
            ask.append(f"{wide * N} {K} {M} linear"), expect.append(dw)
    got = plans(tmp_path, ask)
    assert len(got) == len(ask)
    for line, want, (large, whole_, rest, parts) in zip(ask, expect, got):
        assert bool(large) == (want is not None), line
        if want is not None:
            assert whole_ >= 192 and (rest > 0 and parts > 1) == want, line
    pairs = plans(tmp_path, [f"{M} {wide * N} {K} pair" for sizes, wide in ((BACKWARD, 1), (GATED_BACKWARD, 2))
                             for M, N, K, *_ in sizes])
    assert all(p == [0] for p in pairs)     # large products are launches of their own


class Space:
    """A workspace between guard elements."""

    def __init__(self, n):
        assert n % 4 == 0
        self.out = Out(1, n // 4, F)
        self.t = self.out.vector().view(torch.uint8) if n else None

    def check(self):
        guard = torch.cat([self.out.bits[:self.out.lo], self.out.bits[self.out.hi:]])
        assert bool((guard == self.out.mark).all()), "wrote outside the workspace"


@pytest.mark.gpu
@pytest.mark.parametrize("size", FORWARD, ids=ids)
def test_linear(size):
    M, N, K, pad, _ = size
    gen = generator(M + N + K)
    x, w = whole(gen, M, K, 3, pad), whole(gen, N, K, 3, pad)
    b, r = whole(gen, 1, N, 8)[0], whole(gen, M, N, 8, pad)
    out, z, ws = Out(M, N, F, pad), Out(M, N, F, pad), Space(T.taco_linear_workspace_bytes(M, N, K))
    T.taco_linear(x, w, out.t, bias=b, act=RELU, residual=r, preact=z.t, workspace=ws.t)
    torch.cuda.synchronize()
    out.check("out")
    z.check("preact")
    ws.check()
    want = x.double() @ w.double().t() + b.double()
    assert torch.equal(z.t.double(), want)
    assert torch.equal(out.t.double(), want.clamp(min=0) + r.double())
    plain = Out(M, N, BF, pad)
    T.taco_linear(x, w, plain.t, workspace=ws.t)
    torch.cuda.synchronize()
    plain.check("plain")
    assert torch.equal(plain.t, (want - b.double()).to(BF))


@pytest.mark.gpu
@pytest.mark.parametrize("size", GATED, ids=ids)
def test_gated(size):
    M, N, K, pad, _ = size
    gen = generator(M + N + K)
    x, w = whole(gen, M, K, 1, pad), whole(gen, 2 * N, K, 1, pad)
    out, z, ws = Out(M, N, F, pad), Out(M, 2 * N, F, pad), Space(T.taco_gated_linear_workspace_bytes(M, N, K))
    T.taco_gated_linear(x, w, out.t, act=RELU, preact=z.t, workspace=ws.t)
    torch.cuda.synchronize()
    out.check("out")
    z.check("preact")
    ws.check()
    want = x.double() @ w.double().t()
    assert torch.equal(z.t.double(), want)
    assert torch.equal(out.t.double(), want[:, :N].clamp(min=0) * want[:, N:])


@pytest.mark.gpu
@pytest.mark.parametrize("size", BACKWARD, ids=ids)
def test_linear_backward(size):
    M, N, K, pad = size[:4]
    gen = generator(M + N + K)
    x, w = whole(gen, M, K, 3, pad), whole(gen, N, K, 3, pad)
    d, z = whole(gen, M, N, 3, pad), whole(gen, M, N, 2, pad)
    ws = Space(T.taco_linear_backward_workspace_bytes(M, N, K))
    for act in (NONE, RELU):
        dx, dw, db = Out(M, K, F, pad), Out(N, K, F, pad), Out(1, N, F)
        T.taco_linear_backward(d, x, w, act=act, preact=z if act else None, dx=dx.t, dw=dw.t, dbias=db.vector(),
                               workspace=ws.t)
        torch.cuda.synchronize()
        for o, n in ((dx, "dx"), (dw, "dw"), (db, "dbias")):
            o.check(n)
        ws.check()
        dz = d.double() * slope64(z.double(), act)
        assert torch.equal(dx.t.double(), dz @ w.double()), act
        assert torch.equal(dw.t.double(), dz.t() @ x.double()), act
        assert torch.equal(db.vector().double(), dz.sum(0)), act


@pytest.mark.gpu
@pytest.mark.parametrize("size", GATED_BACKWARD, ids=ids)
def test_gated_backward(size):
    M, N, K, pad = size[:4]
    gen = generator(M + N + K)
    x, w = whole(gen, M, K, 2, pad), whole(gen, 2 * N, K, 2, pad)
    d, z = whole(gen, M, N, 2, pad), whole(gen, M, 2 * N, 2, pad, dtype=F)
    dx, dw = Out(M, K, F, pad), Out(2 * N, K, BF, pad)
    ws = Space(T.taco_gated_linear_backward_workspace_bytes(M, N, K))
    T.taco_gated_linear_backward(d, x, w, act=RELU, preact=z, dx=dx.t, dw=dw.t, workspace=ws.t)
    torch.cuda.synchronize()
    dx.check("dx")
    dw.check("dw")
    ws.check()
    d64, g, u = d.double(), z[:, :N].double(), z[:, N:].double()
    dz = torch.cat([d64 * u * slope64(g, RELU), d64 * act64(g, RELU)], 1)
    assert torch.equal(dx.t.double(), dz @ w.double())
    assert torch.equal(dw.t, (dz.t() @ x.double()).to(BF))


@pytest.mark.gpu
def test_calls_allocate_nothing():
    """Once a kernel has been loaded, a call leaves the device's free memory
    as it was (torch's own allocations are made before)."""
    gen = generator(21)
    M, N, K = 4100, 1032, 1048
    x, w, d, z = whole(gen, M, K, 2), whole(gen, 2 * N, K, 2), whole(gen, M, N, 2), whole(gen, M, 2 * N, 2)
    h, y, stat = torch.empty_like(d), torch.empty_like(x), torch.zeros(2, M, device="cuda") + 1
    dx, dw, db, g = torch.empty_like(x), torch.empty_like(w), torch.empty(2 * N, device="cuda"), torch.empty(2, K, device="cuda")
    sizes = (T.taco_linear_workspace_bytes(M, 2 * N, K), T.taco_linear_backward_workspace_bytes(M, 2 * N, K),
             T.taco_gated_linear_workspace_bytes(M, N, K), T.taco_gated_linear_backward_workspace_bytes(M, N, K),
             T.taco_layer_norm_backward_workspace_bytes(M, K))
    ws = torch.empty(max(sizes), dtype=torch.uint8, device="cuda")

    def calls():
        T.taco_layer_norm(x, None, None, 1e-5, y, mean=stat[0], rstd=stat[1])
        T.taco_layer_norm_backward(x, y, None, stat[0], stat[1], dx=dx, dweight=g[0], dbias=g[1], workspace=ws)
        T.taco_linear(x, w, z, act=GELU, workspace=ws)
        T.taco_linear_backward(z, x, w, act=GELU, preact=z, dx=dx, dw=dw, dbias=db, workspace=ws)
        T.taco_gated_linear(x, w, h, preact=z, workspace=ws)
        T.taco_gated_linear_backward(d, x, w, preact=z, dx=dx, dw=dw, workspace=ws)
        torch.cuda.synchronize()

    calls()
    free = torch.cuda.mem_get_info()[0]
    calls()
    assert torch.cuda.mem_get_info()[0] == free
