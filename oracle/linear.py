"""Float64 restatement of y = act(x w^T + bias) + residual, and how far a float32 evaluation may be from it.

TEST INFRASTRUCTURE ONLY (see the package docstring).  Pins: ``tests/test_oracle_linear.py``.
"""

import math

import numpy as np

_erfc = np.vectorize(math.erfc, otypes=[np.float64])


def activate(v, name):
    with np.errstate(over="ignore"):
        if name == "relu":
            return np.maximum(v, 0.0)
        if name == "silu":
            return v / (1.0 + np.exp(-v))
        if name == "gelu":
            return 0.5 * v * _erfc(-v / math.sqrt(2.0))
        if name == "gelu_tanh":
            return v / (1.0 + np.exp(-2.0 * math.sqrt(2.0 / math.pi) * (v + 0.044715 * v ** 3)))
        if name == "sigmoid":
            return 1.0 / (1.0 + np.exp(-v))
    return v


def linear(x, w, bias=None, activation=None, residual=None):
    v = x @ w.T
    if bias is not None:
        v = v + bias
    v = activate(v, activation)
    return v if residual is None else v + residual


def bound(x, w, bias=None, activation=None, residual=None, eps=2.0 ** -24, tiny=0.0):
    """Largest error of y in a type whose rounding is off by at most ``eps`` of the value (2**-8 bf16, 2**-11 fp16,
    2**-24 float32) or ``tiny`` (half its smallest step): the tensor core rounds its running sum at most four times
    per 16 values of K, each by 2**-24 of the sum of magnitudes; no activation's slope is above 1.13; bias, activation and
    residual take a few float32 roundings of their results."""
    mag = np.abs(x) @ np.abs(w).T
    v = x @ w.T
    if bias is not None:
        v, mag = v + bias, mag + np.abs(bias)
    err = 1.13 * (x.shape[1] / 4 + 16) * 2.0 ** -24 * mag
    a = activate(v, activation)
    err = err + 2.0 ** -20 * np.abs(a) + 2.0 ** -119
    y = a if residual is None else a + residual
    return err + eps * (np.abs(y) + err) + tiny
