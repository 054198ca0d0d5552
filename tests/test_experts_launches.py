"""The launches that calls of the products by group make, without a GPU: the
entry points and plans as they are, with a recorder in place of the launch (see
experts_launches.cpp). At every size that the entry points accept, a launch stays
below 2^32 threads along each axis and within a CU's LDS."""

import os
import subprocess

import pytest

from tests.conftest import ROOT
from tests.test_layers_large import HIPCC

CALLS = ("linear", "gated", "linear-dx", "linear-dw", "linear-both", "linear-db", "linear-all", "gated-dx", "gated-dw",
         "gated-both")
MOST = 1 << 35          # elements of a tensor
DIM = 1 << 20           # of N, 2 F and K


@pytest.fixture(scope="session")
def launches(tmp_path_factory):
    if not os.path.exists(HIPCC):
        pytest.skip("hipcc not installed")
    import importlib.util
    spec = importlib.util.spec_from_file_location(
        "taco_build", os.path.join(ROOT, "quantized_compression_tensor_amd", "build.py"))
    build = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(build)
    exe = str(tmp_path_factory.mktemp("launches") / "experts_launches")
    flags = [f for f in build.FLAGS if f != "-O3"]
    b = subprocess.run([HIPCC, *flags, "-O1", "-x", "hip", f"-I{build.CSRC}",
                        os.path.join(ROOT, "tests", "experts_launches.cpp"), "-o", exe],
                       capture_output=True, text=True, timeout=900)
    assert b.returncode == 0, b.stderr[-3000:]

    def ask(lines):
        """Of each (call, groups, M, N, K, offset): the status, and (kernel, grid x, grid y, threads, LDS) of its launches."""
        text = "".join(" ".join(map(str, line)) + "\n" for line in lines)
        r = subprocess.run([exe], input=text, capture_output=True, text=True, timeout=120)
        assert r.returncode == 0
        out = [line.split("\t") for line in r.stdout.splitlines()]
        assert len(out) == len(lines)
        return [(int(o[0]), [(p.split("|")[0], *map(int, p.split("|")[1:])) for p in o[1:]]) for o in out]
    return ask


def sizes():
    """The largest N for each number of groups and rows to a group, and the largest K for that N; and the other way round."""
    for groups in (1, 7, 33, 64, 65, 512, 777, 1000, 1024):
        for per in (1, 4, 5, 31, 32, 33, 34, 40, 63, 64, 65, 66, 127, 128, 129, 255, 256, 257, 300, 4096, 1 << 20):
            for rows in {per * groups, per * groups + groups - 1}:
                if rows > 1 << 30:
                    continue
                for most in {min(DIM, MOST // rows), min(DIM, MOST // rows) // 2 + 1}:
                    other = min(DIM, MOST // (groups * most), MOST // rows)
                    for less in {other, min(other, 64), 1}:
                        if less > 0:
                            yield groups, rows, most, less
                            yield groups, rows, less, most


def test_launches_at_the_largest_sizes(launches):
    lines = [(call, groups, rows, max(1, n // (2 if call.startswith("gated") else 1)), k, offset)
             for groups, rows, n, k in sizes() for call in CALLS for offset in (0, 1)]
    # dx of 33 to 64 rows to a group, in tall tiles: more threads than a launch has
    lines += [(call, 1024, rows, 32, k, 0) for rows, k in ((33792, 1016800), (40960, 838860))
              for call in ("linear-dx", "linear-all")]
    accepted = 0
    for line, (status, all_) in zip(lines, launches(lines)):
        # (the largest tensors with their rows further apart than their columns are too large)
        assert status == 0 or line[-1] > 0, line
        accepted += status == 0
        assert all_ or status, line
        for kernel, x, y, threads, lds in all_:
            if kernel.startswith("k_"):
                assert 0 < x and x * threads < 1 << 32 and 0 < y < 1 << 16 and lds <= 160 * 1024, (line, kernel, x, y)
    assert accepted > len(lines) // 2


def test_every_kernel_is_run_by_a_test(launches):
    """The kernels (with their tiles) that calls of any sizes take are those that
    the cases of test_experts.py and test_experts_gradients.py take."""
    import random

    from tests.test_experts import CASES, REAL
    from tests.test_experts_gradients import LARGE, ONE_BY_ONE, half

    def line(call, c):
        return call, c.G, c.M, c.N, c.K, int(bool(c.pad or c.offset))

    def kernels(lines):
        return {k for _, all_ in launches(lines) for k, *_ in all_}

    cases = [line(call, c) for c in CASES + REAL if c.M for call in ("linear", "gated", "linear-all", "gated-both")]
    cases += [line(call, c) for c in ONE_BY_ONE for call in ("linear-dx", "linear-dw", "linear-db", "linear-both")]
    cases += [line(call, half(c)) for c in ONE_BY_ONE for call in ("gated-dx", "gated-dw", "gated-both")]
    cases += [line("linear-all", c) for c in LARGE]
    rng, lines = random.Random(3), []
    for _ in range(100000):
        groups, rows, n, k = rng.choice([1, 2, 3, 8, 16, 40, 64, 65, 300]), *(int(2 ** rng.uniform(0, e)) for e in (18, 14, 14))
        offset = rng.randint(0, 1)
        if not offset:
            n, k = -(-n // 8) * 8, -(-k // 8) * 8
        lines.append((rng.choice(CALLS), groups, rows, n, k, offset))
    assert kernels(lines) <= kernels(cases), kernels(lines) - kernels(cases)
    large = "taco::Tiles<256, 256, 2, 4>"
    both = f"k_experts_back<{large}, {large}, false, false>"
    took = [{k for k, *_ in all_} for _, all_ in launches([line("linear-all", c) for c in LARGE])]
    assert [both in t for t in took] == [True] * 5 + [False] * 4
    for t in took[5:7] + took[8:]:      # of dw alone
        assert any(k.startswith(f"k_experts_dw<{large}") for k in t)
    assert f"k_experts<{large}, true, false, false>" in took[7]


def test_tiles_are_enough_for_any_rows(launches):
    """The workgroups of a launch are enough for every distribution of the rows
    over the groups: full tiles, and for the rows left tiles half as high (32 rows:
    as high). Among them the worst: as many groups as there can be with one row
    more than a half, or one."""
    import random
    import re
    rng, lines = random.Random(8), []
    for _ in range(400):
        groups, per = rng.choice([1, 2, 3, 8, 33, 64, 100, 300]), rng.choice([5, 20, 33, 50, 64, 70, 200, 256, 300, 700])
        rows = per * groups + rng.randrange(groups)
        n, k = rng.choice([120, 520, 2056, 8200]), rng.choice([72, 264, 2056, 6000])
        lines.append((rng.choice(["linear", "gated", "linear-dx", "gated-dx"]), groups, rows, n, k, rng.randint(0, 1)))
    seen = set()
    for (call, groups, rows, n, k, _), (status, all_) in zip(lines, launches(lines)):
        assert status == 0
        tiles = {kernel.split("<")[0]: (kernel, x) for kernel, x, *_ in all_}
        if "k_experts" not in tiles:      # few rows: a workgroup takes all of a group's
            continue
        kernel, workgroups = tiles["k_experts"]
        have = tiles["k_experts_join"][1] if "k_experts_join" in tiles else workgroups      # (K cut: parts of each)
        height, width = map(int, re.search(r"Tiles<(\d+), (\d+)", kernel).groups())
        columns = -(-k // width) if call.endswith("-dx") else -(-n // (width // 2 if call == "gated" else width))
        low = max(32, height // 2)
        seen.add((height, call.endswith("-dx")))
        ways = [[rows // groups + (g < rows % groups) for g in range(groups)], [rows] + [0] * (groups - 1)]
        for least in (1, low + 1, height + 1, height + low + 1):
            used = min(groups, rows // least)
            ways.append([least] * used + [rows - least * used] if used < groups else [least] * (used - 1) + [rows - least * (used - 1)])
        for _ in range(20):
            cuts = sorted(rng.choice([0, rows, rng.randint(0, rows)]) for _ in range(groups - 1))
            ways.append([b - a for a, b in zip([0] + cuts, cuts + [rows])])
        for way in ways:
            assert sum(way) == rows and len([s for s in way if s]) <= groups
            need = sum(s // height + -(-(s % height) // low) for s in way) * columns
            assert need <= have, (call, groups, rows, n, k, kernel, way)
    assert seen == {(h, dx) for h in (32, 64, 128, 256) for dx in (False, True)}
