"""Float64 restatement of a whole MoE layer on given weights ("GEMM 执行方式" §4.2-§4.4, with the activation between
the two products) and how far a float32 evaluation with split operands may be from it.

Weights are float64 matrices (dequantised codes, or bf16 values): w13 [E, 2 I, K] (gate rows, up rows), w2 [E, K, I].

TEST INFRASTRUCTURE ONLY (see the package docstring).  Pins: ``tests/test_oracle_few_tokens.py``.
"""

import numpy as np


def _silu(g):
    return g / (1.0 + np.exp(-g))


def _expert(x, w13, w2):
    y = x @ w13.T
    g, u = np.split(y, 2, axis=1)
    return g, u, _silu(g) * u


def few_token_moe(x, ids, weights, w13, w2, shared=None, addend=None):
    """z float64 [T, K]; ids outside [0, E) take no expert; an expert named twice counts with both weights."""
    z = np.zeros_like(x)
    for t in range(x.shape[0]):
        for e, p in zip(ids[t], weights[t]):
            if 0 <= e < w13.shape[0]:
                z[t] += float(p) * (_expert(x[t:t + 1], w13[e], w2[e])[2] @ w2[e].T)[0]
    if shared is not None:
        z += _expert(x, *shared)[2] @ shared[1].T
    return z if addend is None else z + addend


def bound(x, ids, weights, w13, w2, shared=None, addend=None, fp8=True, terms=2):
    """Largest error of z before its rounding to bf16 (half a step, 2**-8 |z|, comes on top).

    First product: the tensor core rounds the running sum at most four times per instruction (32 values of E4M3, 16 of
    bf16), each by 2**-24 of the sum of magnitudes; E4M3 weights meet x as two terms (two such sums), off by 2**-21
    of the largest of the 128 values.  Then |d silu| <= 1.1 |dg|, a few float32 roundings, the split of
    p h into ``terms`` terms and the second product's sum over all experts of the token.  An E4M3 term is off by half a
    step of its 4 significant bits, and what is left is at most half a step of the leading one: 2**-9 of a value with two terms,
    2**-14 with three, or, where the last term is subnormal, half of 2**-9 / 16**(terms - 1) of a block whose largest
    is above 224: 2**-21 and 2**-25 of that.  bf16 terms hold 8 bits: 2**-8 of a value with one, 2**-17 with two.
    Values of h and z below the normal range, 2**-126, may count as 0."""
    T, K = x.shape
    steps = 4 / (32 if fp8 else 16) * 2.0 ** -24 * (2 if fp8 else 1)

    split = {1: 2.0 ** -4, 2: 2.0 ** -9, 3: 2.0 ** -14}[terms] if fp8 else {1: 2.0 ** -8, 2: 2.0 ** -17}[terms]

    def tail(v, n=2):
        if not fp8:
            return np.zeros_like(v)
        blocks = np.abs(v).reshape(v.shape[0], -1, 128)
        return np.repeat(blocks.max(2) * 2.0 ** (-13 - 4 * n), 128, axis=1)

    def expert(rows, a13, a2, p):
        """(error of p W2 h, its sum of magnitudes) for rows of x."""
        g, u, h = _expert(rows, a13, a2)
        m = np.abs(rows) @ np.abs(a13).T * (K * steps) + tail(rows) @ np.abs(a13).T
        dg, du = np.split(m, 2, axis=1)
        dh = 1.1 * dg * (np.abs(u) + du) + np.abs(_silu(g)) * du + 2.0 ** -20 * np.abs(h)
        ph, dh = p * np.abs(h), p * dh
        dh += split * (ph + dh) + tail(ph + dh, terms) + 2.0 ** -126
        return dh @ np.abs(a2).T, ph @ np.abs(a2).T

    err, mag = np.zeros((T, K)), np.zeros((T, K))
    inner = np.zeros(T)
    for t in range(T):
        for e in sorted(set(ids[t])):
            if 0 <= e < w13.shape[0]:
                p = abs(sum(float(q) for k, q in zip(ids[t], weights[t]) if k == e))
                d, m = expert(x[t:t + 1], w13[e], w2[e], p)
                err[t] += d[0]
                mag[t] += m[0]
                inner[t] += w2.shape[2]
    if shared is not None:
        d, m = expert(x, shared[0], shared[1], 1.0)
        err, mag, inner = err + d, mag + m, inner + shared[1].shape[1]
    if addend is not None:
        mag = mag + np.abs(addend)
    return err + (inner[:, None] * steps + 16 * 2.0 ** -24) * mag + 2.0 ** -126
