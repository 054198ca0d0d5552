"""The products' kernels hand LDS stages over by counting accesses under way
(s_waitcnt with a number other than zero), which holds only while the compiled
main loop has the accesses that the source counts: this compiles the kernels
for gfx950 and looks. No GPU needed."""

import importlib.util
import os
import re
import subprocess

import pytest

from tests.conftest import ROOT

HIPCC = "/opt/rocm/bin/hipcc"
LAYERS = os.path.join(ROOT, "quantized_compression_tensor_amd", "csrc_layers")


def compiled(source, folder):
    if not os.path.exists(HIPCC):
        pytest.skip("hipcc not installed")
    spec = importlib.util.spec_from_file_location(
        "taco_build", os.path.join(ROOT, "quantized_compression_tensor_amd", "build.py"))
    build = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(build)
    out = str(folder / "out.s")
    subprocess.run([HIPCC, *build.FLAGS, "--offload-device-only", "-S", os.path.join(LAYERS, source), "-o", out],
                   check=True, capture_output=True, timeout=600)
    return open(out).read()


@pytest.fixture(scope="module")
def assembly(tmp_path_factory):
    return compiled("linear.hip", tmp_path_factory.mktemp("asm"))


def kernels(text, name):
    """(template arguments as mangled, lines) of each kernel called `name`."""
    for m in re.finditer(rf"^(_ZN4taco\d+{name}I\S*):\s*;", text, re.M):
        body = text[m.end():text.index("s_endpgm", m.end())]
        yield m.group(1), body.splitlines()


def main_loops(lines):
    """Instruction lists of the blocks that hold two barriers and products."""
    block = []
    for line in lines + [".LBB_end:"]:
        if re.match(r"\.LBB", line):
            if sum("s_barrier" in i for i in block) >= 2 and any("v_mfma" in i for i in block):
                yield block
            block = []
        elif re.match(r"\s+[a-z]", line):
            block.append(line.strip())


def check_loop(loop, a_by_k, b_by_k, large):
    rows, cols = (8, 4) if large else (4, 4)    # MFMA tiles of a wave
    free_a, free_b = rows // 4, rows // 2       # tiles after which a stage is handed back
    a_reads, b_reads = (2 if a_by_k else 1), (2 if b_by_k else 1)    # LDS reads of an operand
    loads = 8                                   # of a thread in a step: four of each operand
    first, second = [n for n, i in enumerate(loop) if i.startswith("s_barrier")]

    def count(prefix, start, end):
        return sum(i.startswith(prefix) for i in loop[start:end])

    def wait_before(n):
        """The counters that the waits right before barrier n leave."""
        left = {"vmcnt": 63, "lgkmcnt": 15}
        for i in loop[max(0, n - 12):n]:
            if i.startswith("s_waitcnt"):
                for c, v in re.findall(r"(vmcnt|lgkmcnt)\((\d+)\)", i):
                    left[c] = min(left[c], int(v))
        return left

    # b's second half is read, then free_b operands of a, and the wait lets at
    # most the latter be under way
    assert count("ds_read", 0, first) == cols * b_reads + free_b * a_reads
    assert wait_before(first)["lgkmcnt"] <= free_b * a_reads
    # a's stage: the other operands are read before the second barrier, which
    # waits for all of them and for all loads but those of a step
    assert count("ds_read", first, second) == (rows - free_b) * a_reads
    assert wait_before(second)["lgkmcnt"] == 0 and wait_before(second)["vmcnt"] <= loads
    # the loads of a step, half after either barrier
    assert count("buffer_load", 0, first) == 0
    assert count("buffer_load", first, second) == loads // 2
    assert count("buffer_load", second, len(loop)) == loads // 2
    assert not any("lds" not in i for i in loop if i.startswith("buffer_load"))
    # next step's first half
    assert count("ds_read", second, len(loop)) == rows * a_reads + cols * b_reads
    assert free_a < rows and not any(i.startswith(("scratch_", "buffer_store", "global_")) for i in loop)


def test_products_hand_over_what_they_count(assembly):
    seen = 0
    for symbol, lines in kernels(assembly, "k_gemm"):
        tile, flags = re.match(r".*TilesILi(\d+)E.*EE((?:Lb[01]E)+)E", symbol).groups()
        a_by_k, b_by_k, _ = [f == "1" for f in re.findall(r"Lb([01])E", flags)]
        loops = list(main_loops(lines))
        assert len(loops) == 1, symbol
        check_loop(loops[0], a_by_k, b_by_k, tile == "256")
        seen += 1
    assert seen == 8
    for symbol, lines in kernels(assembly, "k_gemm_pair"):
        body = assembly[assembly.index(symbol + ":"):]
        loops = list(main_loops(body[:body.index(".Lfunc_end")].splitlines()))
        assert len(loops) == 2
        for loop in loops:
            by_k = sum(i.startswith("ds_read_b64_tr") for i in loop), sum(i.startswith("ds_read_b128") for i in loop)
            check_loop(loop, by_k[1] == 0, True, False)
        seen += 1
    assert seen == 9


def test_no_kernel_spills(assembly, tmp_path):
    """Registers that do not fit cost more than they save, and in divergent
    code a spilled one has come back wrong."""
    for text in (assembly, compiled("norm.hip", tmp_path)):
        spills = re.findall(r"\.vgpr_spill_count:\s*(\d+)", text)
        assert spills and set(spills) == {"0"}
