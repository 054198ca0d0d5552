"""Norms whose workgroups hold one row at a time and walk over several: more
rows than workgroups at 5120 columns, and beyond 8192 columns, where a lane
takes two steps and the sums over rows have a kernel of their own. The checks
and tolerances are those of test_layers_norm.py (an element of dweight or dbias
is summed over ceil(rows / 512) rows of a workgroup there)."""

import pytest

from tests.layers_util import generator, matrix
from tests.test_layers_norm import BF, EPS, F, check_backward, check_forward

pytestmark = pytest.mark.gpu

SHAPES = [(1100, 5120, BF), (1537, 5121, F), (1100, 8193, F), (2100, 8200, BF), (1100, 16384, BF), (1025, 16379, F)]


@pytest.mark.parametrize("rows,cols,dtype", SHAPES)
def test_forward(rows, cols, dtype):
    gen = generator(rows + cols)
    x = matrix(gen, rows, cols, dtype, mean=0.3)
    weight, bias = matrix(gen, 1, cols, dtype, mean=1.0, sigma=0.2)[0], matrix(gen, 1, cols, F, sigma=0.2)[0]
    check_forward(x, weight, bias, EPS, dtype, 0, 0, f"{rows}x{cols}")


@pytest.mark.parametrize("want", [("dx", "dweight", "dbias"), ("dweight", "dbias"), ("dx",)])
@pytest.mark.parametrize("rows,cols,dtype", SHAPES)
def test_backward(rows, cols, dtype, want):
    check_backward(generator(rows * 3 + cols), rows, cols, dtype, dtype, dtype, 0, 0, f"{rows}x{cols} {want}", want=want)
