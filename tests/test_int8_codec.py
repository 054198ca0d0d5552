"""Rows of 64 elements as codes of taco_quantize_rows and as blocks of the codec
INT8_SYM: the same scales, and codes that differ by one at most, and only next to
a half.

Both multiply x by 127 / A, A = max |x|: the codec with one rounding in the
multiplier (U32 = 2^-24 of its value), the rows with two, and either with one more
in the product. |x 127 / A| is at most 127, so the values that are rounded to whole
numbers lie within 127 (3 U32 + 4 U32^2) of it (the bound 127 * 3.01 * U32), and
rounding can only differ where a half is as near as that."""

import numpy as np
import pytest

import oracle
from oracle import codecs as cd

U32 = 2.0 ** -24


def block_rows(kind, rows=4096):
    """bf16 rows of 64, as float32."""
    rng = np.random.default_rng(11)
    x = rng.standard_normal((rows, 64)).astype(np.float32)
    if kind == "scales":      # A from 2^-95 to 2^126
        x *= np.exp2(rng.integers(-95, 123, (rows, 1))).astype(np.float32)
    elif kind == "halves":    # whole and half numbers: many products next to a half
        x = (rng.integers(-254, 255, (rows, 64)) / 2).astype(np.float32) * np.exp2(rng.integers(-20, 20, (rows, 1))).astype(np.float32)
    return oracle.bf16_bits_to_f32(bf16_bits(x)).reshape(rows, 64)


def bf16_bits(x):
    """To bf16, ties to even (no NaN here)."""
    b = np.ascontiguousarray(x, np.float32).view(np.uint32)
    return ((b + 0x7FFF + ((b >> 16) & 1)) >> 16).astype(np.uint16)


def check(x, rows_codes, rows_scale, block_codes, block_scale):
    """How many codes differ, all of them as documented."""
    assert np.array_equal(rows_scale.view(np.uint32), block_scale.view(np.uint32))
    a, b = rows_codes.astype(int).reshape(x.shape), block_codes.astype(int).reshape(x.shape)
    t = x.astype(np.float64) * 127 / np.abs(x.astype(np.float64)).max(1, keepdims=True)
    for q in (a, b):
        assert np.abs(q - t).max() <= 0.5 + 127 * 3.01 * U32
    apart = a != b
    assert np.abs(a - b).max() <= 1
    assert np.abs(np.abs(t - np.floor(t)) - 0.5)[apart].max(initial=0) <= 127 * 3.01 * U32
    return int(apart.sum())


@pytest.mark.parametrize("kind", ["normal", "scales", "halves"])
def test_definitions(kind):
    from tests.test_int8 import quantized
    import torch
    x = block_rows(kind)
    q, s = quantized(torch.from_numpy(x))
    ref = oracle.compress(cd.Codec.int8_sym(), bf16_bits(x))
    differ = check(x, q, s, ref.codes.view(np.int8), ref.scale)
    if kind == "normal":      # they are not the codec's: 3.9e-4 of them
        assert 0 < differ < 1e-3 * x.size


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["normal", "scales", "halves"])
def test_kernels(kind):
    import torch

    import quantized_compression_tensor_amd as T
    from tests.gpu_util import DEV, gpu_compress, parse
    x = block_rows(kind)
    rows = x.shape[0]
    bits = bf16_bits(x)
    oc = cd.Codec.int8_sym()
    block = parse(gpu_compress(oc, bits)[0], oc, rows, 64)
    q, s = torch.empty(rows, 64, dtype=torch.int8, device=DEV), torch.empty(rows, device=DEV)
    T.taco_quantize_rows(torch.from_numpy(bits.view(np.int16)).to(DEV).view(torch.bfloat16), q, s)
    torch.cuda.synchronize()
    check(x, q.cpu().numpy(), s.cpu().numpy(), block["codes"].view(np.int8), block["scale"])
