"""The row limits that include/taco.h states are the ones that the library has
(workspace sizes need no GPU: 0 is a size that is refused)."""

import os
import re

import quantized_compression_tensor_amd as T
from tests.conftest import ROOT


def stated(pattern):
    text = re.sub(r"\s*\n \*\s*", " ", open(os.path.join(ROOT, "include", "taco.h")).read())
    return 1 << int(re.search(pattern, text).group(1))


def test_rows_of_a_projection():
    most = stated(r"M at most 2\^(\d+) \(TACO_ERR_INVALID_ARG\)")
    for size in (T.taco_linear_backward_workspace_bytes, T.taco_gated_linear_backward_workspace_bytes):
        assert size(most, 8, 8) > 0 and size(most + 1, 8, 8) == 0


def test_rows_of_a_norm():
    end = stated(r"rows below 2\^(\d+) \(TACO_ERR_INVALID_ARG\)")
    size = T.taco_layer_norm_backward_workspace_bytes
    assert size(end - 1, 16) > 0 and size(end, 16) == 0
    assert size((1 << 35) // 16384, 16384) > 0 and size((1 << 35) // 16384 + 1, 16384) == 0
