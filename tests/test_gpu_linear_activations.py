"""linear's activations relative to their size, on sums that are the bias alone, with a tolerance for each of them."""

import numpy as np
import pytest
import torch

import oracle
from block_scaled_fp8_route_gb300 import ops
from tests.gpu_util import require_gpu

pytestmark = pytest.mark.gpu


def tolerance(act, v):
    """Relative error, in units of 2**-24 (a rounding).  exp2 and a quotient are off by 2 steps of 2**-23 each, 8 in all.

    exp(-v): its argument times log2(e) is rounded once and the constant is, which is 2 |v| of the result; then 1 + exp, 1.
    gelu: v^2 / 2 with two roundings and that of a constant, 3 v^2 / 2 of exp(-v^2 / 2).  The fit is off by 4.5e-8 (0.8) and
    its nine steps by half a unit each of sums of up to 0.6 where the result is 0.17 or more (at most 9 * 0.6 / 0.17 = 32); t's
    quotient moves the product by no more than 4; products and the last fma 4.  (max(v, 0) - |v| e loses nothing: for v > 0 it is
    at least |v| e.)
    gelu_tanh: u2 = v (c1 + c2 v v), two constants and four roundings, 6 |u2|, and exp's 2 |u2|."""
    if act == "relu":
        return np.zeros_like(v)
    if act in ("silu", "sigmoid"):
        return 2 * np.abs(v) + 9
    if act == "gelu":
        return 1.5 * v ** 2 + 8 + 1 + 32 + 4 + 4
    return 8 * np.abs(1.5957691216057308 * v + 0.07135481627364643 * v ** 3) + 9


@pytest.mark.parametrize("T", [6, 700])
@pytest.mark.parametrize("act", ["relu", "silu", "gelu", "gelu_tanh", "sigmoid"])
@pytest.mark.parametrize("reach", [1.0, 16.0, 60.0])
def test_relative_to_their_size(act, T, reach):
    dev = require_gpu()
    N = 2048
    x, w = torch.zeros(T, 64, dtype=torch.bfloat16, device=dev), torch.zeros(N, 64, dtype=torch.bfloat16, device=dev)
    bias = torch.linspace(-reach, reach, N, device=dev)
    y = ops.linear(x, w, bias=bias, activation=act, out_dtype=torch.float32).double().cpu().numpy()
    assert ops.device_error() == 0
    v = bias.double().cpu().numpy()
    ref = oracle.linear.activate(v, act)
    # (a quotient by more than 2**126, or an exp below 2**-126, is 0: at most 60 * 2**-126 of the exact one)
    tol = tolerance(act, v) * 2.0 ** -24 * np.abs(ref) + 2.0 ** -118
    worst = np.max(np.abs(y - ref) / tol)
    assert worst <= 1, f"worst {worst:.2f} times the tolerance"
