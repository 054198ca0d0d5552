"""The polynomial in csrc_layers/linear.hip for the normal distribution's
function, read from the source: the error that its comment states for Q, in
float64 (scipy's erfcx is exp(x^2) erfc(x)), and those of Phi, with the steps of
the device function in float32 (exact reciprocal and exp2, which the device has
to a unit in the last place)."""

import os
import re

import numpy as np
from scipy.special import erfcx, ndtr

from tests.conftest import ROOT

SOURCE = open(os.path.join(ROOT, "quantized_compression_tensor_amd", "csrc_layers", "linear.hip")).read()
BODY = SOURCE[SOURCE.index("TACO_DEV float normal_cdf"):SOURCE.index("TACO_DEV float sigmoid")]
NUMBER = r"(-?\d+\.\d+)f"
COEFFICIENTS = [float(re.search(rf"float q = {NUMBER}", BODY).group(1)),
                *(float(c) for c in re.findall(rf"fmaf\(q, t, {NUMBER}\)", BODY))]
P = float(re.search(rf"kP = {NUMBER}", BODY).group(1))


def stated(pattern):
    comment = re.sub(r"\s*\n// ?", " ", SOURCE[SOURCE.index("// Phi(z), the normal"):SOURCE.index("TACO_DEV float normal_cdf")])
    return float(re.search(pattern, comment).group(1))


def test_polynomial():
    assert len(COEFFICIENTS) == 9
    x = np.linspace(0.0, 9.5, 2_000_001)
    t = 1.0 / (1.0 + np.float64(P) * np.sqrt(2.0) * x)
    q = np.polyval(COEFFICIENTS, t)
    error = np.abs(q * t / erfcx(x) - 1.0).max()
    bound = stated(r"relative error below ([\d.]+e-\d+)")
    assert 0.9 * bound <= error <= bound


def test_phi_in_float32():
    f = np.float32
    z = np.concatenate([np.linspace(-13.0, 13.0, 1_300_001), np.linspace(-1e-3, 1e-3, 20_001)]).astype(f)
    z64 = z.astype(np.float64)
    t = (1.0 / (f(P) * np.abs(z) + f(1)).astype(np.float64)).astype(f)
    q = np.full_like(z, COEFFICIENTS[0])
    for c in COEFFICIENTS[1:]:
        q = (q.astype(np.float64) * t + f(c)).astype(f)          # one rounding, as a fused multiply-add
    e = np.exp2((-(z * z) * f(0.72134752044448170)).astype(np.float64)).astype(f)
    h = f(0.5) * t * q * e
    phi = np.where(z < 0, h, f(1) - h).astype(np.float64)
    want = ndtr(z64)
    assert np.abs(phi - want).max() <= stated(r"Phi is within ([\d.]+e-\d+)")
    inner = np.abs(z64) < 6
    assert (np.abs(phi - want)[inner] / want[inner]).max() <= stated(r"within ([\d.]+e-\d+) of its value for \|z\| < 6")
