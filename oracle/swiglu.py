"""SwiGLU of a gate-up product, and its 1 x 128 quantisation, in float64.

TEST INFRASTRUCTURE ONLY (see the package docstring).

Definition: y = [g | u] of 2 K columns, h = g / (1 + exp(-g)) * u; blocks of
128 along K (the last one may be short, padded with zeros) are quantised as in
``oracle/quantise.py``.

Pins: ``tests/test_oracle_swiglu.py`` (closed forms, oddness identity
silu(x) - silu(-x) = x, equality with the quantiser on bf16-exact inputs).
"""

import numpy as np

from . import formats
from .quantise import BLOCK, _block_exponent


def swiglu(y_bf16_bits):
    """h float64 [T, K] of y [T, 2 K] (bf16 bit patterns)."""
    y = formats.bf16_bits_to_f64(y_bf16_bits)
    K = y.shape[1] // 2
    with np.errstate(over="ignore", invalid="ignore"):
        return y[:, :K] / (1.0 + np.exp(-y[:, :K])) * y[:, K:]


def padded_blocks(h):
    T, K = h.shape
    Kp = (K + BLOCK - 1) // BLOCK * BLOCK
    full = np.zeros((T, Kp))
    full[:, :K] = h
    return full.reshape(T, Kp // BLOCK, BLOCK)


def swiglu_quantise(y_bf16_bits):
    """(q uint8 [T, Kp], sf_bytes uint8 [T, Kp/128])."""
    hb = padded_blocks(swiglu(y_bf16_bits))
    e = _block_exponent(np.max(np.abs(hb), axis=2))
    q = formats.e4m3_encode(np.ldexp(hb, -e[:, :, None]))
    return q.reshape(hb.shape[0], hb.shape[1] * BLOCK), (e + 127).astype(np.uint8)
