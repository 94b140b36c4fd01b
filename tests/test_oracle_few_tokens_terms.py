"""The bound of ``few_token_moe`` by the number of terms that h is split into: an evaluation with that many terms is within
it, one with a term fewer is not, on a layer where the errors of single values of h show."""

import numpy as np
import pytest
import torch

import oracle
from oracle import few_tokens
from tests.few_cases import cancelling
from tests.gpu_util import bits16


def _e4m3(v):
    return oracle.formats.e4m3_decode(oracle.formats.e4m3_encode(v))


def _bf16(v):
    return oracle.formats.bf16_bits_to_f64(oracle.formats.bf16_round(v))


def split(v, terms, fp8):
    """v in blocks of 128 as the sum of its terms: E4M3 with a power of two per block and 2**-4 from term to term, or bf16."""
    rest, got = v.reshape(-1, 128).copy(), 0.0
    scale = 1.0
    if fp8:
        scale = 2.0 ** np.ceil(np.log2(np.maximum(np.abs(rest).max(1, keepdims=True), 1e-30) / 448))
    for k in range(terms):
        step = scale * 16.0 ** -k if fp8 else 1.0
        part = (_e4m3(rest / step) if fp8 else _bf16(rest)) * step
        got, rest = got + part, rest - part
    return got.reshape(v.shape)


def evaluate(x, ids, p, w13, w2, terms, fp8):
    """z in float32 with h split, before its rounding to bf16."""
    z = np.zeros(x.shape, np.float32)
    for t in range(x.shape[0]):
        e, I = ids[t, 0], w2.shape[2]
        y = np.float32(w13[e]) @ np.float32(x[t])
        h = np.float32(p[t, 0]) * (y[:I] / (1 + np.exp(-y[:I])) * y[I:])
        z[t] = w2[e] @ split(h.astype(np.float64), terms, fp8)
    return z


def case(seed):
    return [oracle.formats.bf16_bits_to_f64(bits16(t)) if t.dtype == torch.bfloat16 else t.numpy()
            for t in cancelling(6, seed=seed)]


@pytest.mark.parametrize("fp8,terms", [(True, 2), (True, 3), (False, 2)])
@pytest.mark.parametrize("seed", range(3))
def test_a_term_fewer_is_outside_the_bound(fp8, terms, seed):
    args = case(seed)
    ref = few_tokens.few_token_moe(*args)
    assert np.abs(ref).max() < 1e-12
    tol = few_tokens.bound(*args, fp8=fp8, terms=terms)
    tol = tol + 2.0 ** -8 * tol
    assert np.all(np.abs(evaluate(*args, terms, fp8) - ref) <= tol)
    assert np.mean(np.abs(evaluate(*args, terms - 1, fp8) - ref) > tol) > 0.2


@pytest.mark.parametrize("terms,rel,tail", [(1, 2.0 ** -4, 2.0 ** -17), (2, 2.0 ** -9, 2.0 ** -21), (3, 2.0 ** -14, 2.0 ** -25)])
def test_split_of_float32_values(terms, rel, tail):
    r = np.random.default_rng(terms)
    v = np.float32(r.standard_normal((256, 128)) * np.exp2(r.integers(-30, 1, (256, 128)))).astype(np.float64)
    top = np.abs(v).max(1, keepdims=True)
    err = np.abs(split(v, terms, True) - v)
    assert np.all(err <= np.maximum(rel * np.abs(v), tail * top))
    assert np.max(err / np.abs(v)) > rel / 2                         # (and is not far less)
    one = np.float32(r.standard_normal(4096)).astype(np.float64).reshape(-1, 128)
    assert np.all(np.abs(split(one, terms, False) - one) <= (2.0 ** -8, 2.0 ** -17, 2.0 ** -26)[terms - 1] * np.abs(one))
