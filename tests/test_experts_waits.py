"""As test_layers_waits.py, for the products by group and of 8-bit codes: the
compiled main loops have the accesses that their counted waits rely on, for
each tile, and no kernel spills. No GPU needed."""

import re

import pytest

from tests.test_layers_waits import compiled, kernels, main_loops


@pytest.fixture(scope="module", params=["int8.hip", "experts.hip"])
def assembly(request, tmp_path_factory):
    return request.param, compiled(request.param, tmp_path_factory.mktemp("asm"))


# Rows of a tile: the tile for the rows left by it.
REST = {256: [128, 256, 2, 4], 128: [64, 128, 2, 2], 64: [32, 128, 2, 2], 32: [32, 128, 2, 2]}


def check_loop(loop, tile, a_by_k, b_by_k):
    bm, bn, wgm, wgn = tile
    threads, rows, cols = 64 * wgm * wgn, bm // wgm // 16, bn // wgn // 16
    free_a, free_b = rows // 4, rows // 2
    next_b = free_a + 1 if free_a + 1 < rows else free_a
    a_reads, b_reads = (2 if a_by_k else 1), (2 if b_by_k else 1)
    loads_a, loads_b = bm * 8 // threads, bn * 8 // threads
    first, second = [n for n, i in enumerate(loop) if i.startswith("s_barrier")]

    def count(prefix, start, end):
        return sum(i.startswith(prefix) for i in loop[start:end])

    def wait_before(n):
        left = {"vmcnt": 63, "lgkmcnt": 15}
        for i in loop[max(0, n - 12):n]:
            if i.startswith("s_waitcnt"):
                for c, v in re.findall(r"(vmcnt|lgkmcnt)\((\d+)\)", i):
                    left[c] = min(left[c], int(v))
        return left

    # b's second half and free_b operands of a are read before b's stage is handed back
    assert count("ds_read", 0, first) == cols * b_reads + free_b * a_reads
    assert wait_before(first)["lgkmcnt"] <= free_b * a_reads
    # the rest of a's before its own, with the loads of one step under way at most
    assert count("ds_read", first, second) == (rows - free_b) * a_reads
    assert wait_before(second)["lgkmcnt"] == 0 and wait_before(second)["vmcnt"] <= loads_a + loads_b
    assert count("buffer_load", 0, first) == 0
    assert count("buffer_load", first, second) == loads_b and count("buffer_load", second, len(loop)) == loads_a
    assert not any("lds" not in i for i in loop if i.startswith("buffer_load"))
    assert count("ds_read", second, len(loop)) == rows * a_reads + cols * b_reads and next_b < rows
    assert not any(i.startswith(("scratch_", "buffer_store", "global_")) for i in loop)


def test_products_hand_over_what_they_count(assembly):
    source, text = assembly
    seen = 0
    for name in ("k_int8", "k_experts", "k_experts_dw", "k_experts_back"):
        for symbol, _ in kernels(text, name):
            tiles = [[int(v) for v in t] for t in re.findall(r"ILi(\d+)ELi(\d+)ELi(\d+)ELi(\d+)E", symbol)]
            flags = [f == "1" for f in re.findall(r"Lb([01])E", symbol)]
            body = text[text.index(symbol + ":"):]
            loops = list(main_loops(body[:body.index(".Lfunc_end")].splitlines()))
            # dw reads both operands transposed; forward products neither
            gradient = name == "k_experts" and flags[0]
            # by way of the registers (the first of the gradients' two flags): nothing is counted but dw's
            direct = name != "k_experts_dw" and flags[0 if name == "k_experts_back" else -1]
            few = name == "k_experts_back" and flags[1]       # and there dw's is not either
            dw = [name != "k_experts" and not any(i.startswith("ds_read_b128") for i in l) for l in loops]
            rest = [REST[t[0]] if name in ("k_experts", "k_experts_back") else None for t in tiles[:1]]
            if direct:
                loops = [l for l, is_dw in zip(loops, dw) if is_dw]
                dw = [True] * len(loops)
            expect = {"k_int8": 1, "k_experts_dw": 1, "k_experts": 2, "k_experts_back": 3}[name] - few
            expect -= {"k_int8": 1, "k_experts": 2, "k_experts_back": 2}[name] if direct else 0
            assert len(loops) == expect and sum(dw) == (name in ("k_experts_dw", "k_experts_back")) - few, symbol
            for loop, is_dw in zip(loops, dw):
                # which tile it is of: full ones, those of the rows left (half as high), or dw's
                products = sum(i.startswith("v_mfma") for i in loop)
                choice = [tiles[-1]] if is_dw else [t for t in [tiles[0], *rest] if t and t[0] * t[1] // (t[2] * t[3]) // 128 == products]
                assert choice, symbol
                check_loop(loop, choice[0], is_dw, is_dw or gradient or name == "k_experts_back")
            seen += 1
    assert seen >= 4


def test_no_kernel_spills(assembly):
    spills = re.findall(r"\.vgpr_spill_count:\s*(\d+)", assembly[1])
    assert spills and set(spills) == {"0"}
