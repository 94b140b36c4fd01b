"""The fit of erfc in linear's gelu: how far the coefficients in the source are from it, in 64 bits.  CPU-only."""

import os
import re

import numpy as np
import pytest

from block_scaled_fp8_route_gb300 import build

special = pytest.importorskip("scipy.special")


def test_coefficients():
    with open(os.path.join(build.CSRC, "linear.cu"), encoding="utf-8") as f:
        src = f.read()
    number = r"(-?[0-9.]+)f"
    listed = re.search(r"constexpr float c\[8\] = \{([^}]*)\}", src).group(1)
    c = [float(v) for v in re.findall(number, listed)] + [float(re.search(r"float q0 = " + number, src).group(1))]
    slope = float(re.search(r"fmaf\(a, " + number + r", 1\.f\)", src).group(1))
    assert len(c) == 9
    v = np.linspace(0, 20, 400001)                                   # |v| of gelu(v), the range that it is clamped to
    t = 1 / (1 + np.float64(np.float32(slope)) * v)
    q = np.polynomial.polynomial.polyval(t, np.float64(np.float32(c)))
    off = np.abs(t * q / special.erfcx(v / np.sqrt(2)) - 1).max()
    assert 4.4e-8 < off < 4.6e-8
