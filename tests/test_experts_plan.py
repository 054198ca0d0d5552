"""What experts.hip's host code plans, without a GPU: launches of the largest
sizes stay below 2^32 threads, the tiles counted are enough for any distribution
of the rows, and the sizes of the tests on the GPU take the tiles that they are
there for."""

import os
import random
import subprocess

import pytest

from tests.conftest import ROOT
from tests.test_layers_large import HIPCC


@pytest.fixture(scope="module")
def plans(tmp_path_factory):
    if not os.path.exists(HIPCC):
        pytest.skip("hipcc not installed")
    import importlib.util
    spec = importlib.util.spec_from_file_location(
        "taco_build", os.path.join(ROOT, "quantized_compression_tensor_amd", "build.py"))
    build = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(build)
    exe = str(tmp_path_factory.mktemp("plan") / "experts_plan")
    flags = [f for f in build.FLAGS if f != "-O3"]
    b = subprocess.run([HIPCC, *flags, "-O1", "-x", "hip", f"-I{build.CSRC}", os.path.join(ROOT, "tests", "experts_plan.cpp"),
                        "-o", exe], capture_output=True, text=True, timeout=900)
    assert b.returncode == 0, b.stderr[-3000:]

    def ask(lines):
        """(forward, dx) of each line: tile rows, tiles, parts, threads, threads of the ranges."""
        text = "".join(" ".join(map(str, line)) + "\n" for line in lines)
        r = subprocess.run([exe], input=text, capture_output=True, text=True, timeout=60)
        assert r.returncode == 0
        rows = [[int(v) for v in line.split()] for line in r.stdout.splitlines()]
        assert len(rows) == 2 * len(lines)
        return list(zip(rows[::2], rows[1::2]))
    return ask


def test_largest_launches(plans):
    sizes = [(1024, 32768, 1 << 20, 32), (1024, 65536, 1 << 19, 32), (1024, 131072, 1 << 18, 32), (1, 1 << 30, 32, 32),
             (1024, 1 << 30, 32, 32), (1024, 1 << 30, 1, 1), (1024, 1024, 1 << 20, 32), (1, 32768, 1 << 20, 1 << 15),
             (1024, 262144, 1 << 17, 256), (512, 16384, 1 << 20, 64), (1024, 1, 1 << 20, 32), (33, 1 << 25, 1024, 1024)]
    for size, both in zip(sizes, plans(sizes)):
        for _, tiles, parts, threads, ranges in both:
            assert 0 < tiles and 0 < parts and threads < 1 << 32 and ranges < 1 << 32, size


def test_tiles_are_enough(plans):
    """Full tiles and those of the rows left, half as high (32 rows: as high), of
    random distributions of the rows over the groups."""
    rng = random.Random(4)
    sizes = [(rng.randint(1, 200), rng.randint(1, 20000), 128, 64) for _ in range(60)]
    for (groups, rows, *_), (forward, _) in zip(sizes, plans(sizes)):
        height, tiles = forward[:2]
        half = max(32, height // 2)
        for _ in range(20):
            cuts = sorted(rng.choice([0, rows, rng.randint(0, rows)]) for _ in range(groups - 1))
            sizes_ = [b - a for a, b in zip([0] + cuts, cuts + [rows])]
            need = sum(s // height + -(-(s % height) // half) for s in sizes_)
            assert need <= tiles * (256 if height == 256 else 128) // 128, (groups, rows, height)


def test_shapes_of_the_cases(plans):
    """The cases of test_experts.py take every height of tile, with K whole and cut."""
    from tests.test_experts import CASES
    seen = set()
    for (f, x), c in zip(plans([(c.G, c.M, c.N, c.K) for c in CASES if c.M > 32]), [c for c in CASES if c.M > 32]):
        seen.add((f[0], f[2] > 1))
    assert {h for h, _ in seen} == {32, 64, 128, 256}
    assert (32, True) in seen and (64, True) in seen and (128, True) in seen
