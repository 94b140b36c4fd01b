"""Pins of the block oracle: a token-by-token restatement without routing, masked tokens, the always-active
expert alone."""

import numpy as np
import pytest

import oracle
from oracle import formats, gemm, quantise, swiglu

T, E, K, I, S, KR = 9, 4, 256, 128, 136, 2


def _bits(rng, *shape, scale=1.0):
    return formats.bf16_round(rng.standard_normal(shape) * scale)


@pytest.fixture(scope="module")
def problem():
    rng = np.random.default_rng(5)
    return (_bits(rng, T, K), rng.standard_normal((T, E)), _bits(rng, E, 2 * I, K, scale=0.05),
            _bits(rng, E, K, I, scale=0.05), (_bits(rng, 2 * S, K, scale=0.05), _bits(rng, K, S, scale=0.05)))


def _expert(x_bits, w13, w2):
    """bf16 bits of one expert's output for one token."""
    y = gemm.expert_gemm(*quantise.quantise_act(x_bits[None]), *(v[0] for v in quantise.quantise_weight(w13[None])))
    return gemm.expert_gemm(*swiglu.swiglu_quantise(y), *(v[0] for v in quantise.quantise_weight(w2[None])))[0]


def test_token_by_token(problem):
    x, logits, w13, w2, _ = problem
    z, ids, margin = oracle.block.moe_block(x, logits, w13, w2, KR, sigmoid=True, scale=2.0)
    for t in range(T):
        s = 1 / (1 + np.exp(-logits[t]))
        best = np.argsort(-s)[:KR]
        assert ids[t].tolist() == best.tolist()
        p = (s[best] / s[best].sum() * 2.0).astype(np.float32).astype(np.float64)
        want = sum(p[i] * formats.bf16_bits_to_f64(_expert(x[t], w13[e], w2[e])) for i, e in enumerate(best))
        got = formats.bf16_bits_to_f64(z[t])
        # (float64 products of rows alone and together may differ in a last bit that the bf16 rounding shows)
        assert np.abs(got - want).max() <= 2.0 ** -7 * np.abs(want).max()


def test_the_always_active_expert_alone(problem):
    x, logits, w13, w2, shared = problem
    masked = np.full_like(logits, -np.inf)
    z, ids, _ = oracle.block.moe_block(x, masked, w13, w2, KR)
    assert (ids == -1).all() and not z.any()
    z, _, _ = oracle.block.moe_block(x, masked, w13, w2, KR, shared=shared)
    a = gemm.dequant_rows(*quantise.quantise_act(x))
    y = formats.bf16_bits_to_f64(formats.bf16_round(a @ _dequant(shared[0]).T))
    h = y[:, :S] / (1 + np.exp(-y[:, :S])) * y[:, S:]
    want = h @ _dequant(shared[1])[:, :S].T                # without h's quantisation, within E4M3's step of it
    got = formats.bf16_bits_to_f64(z)
    assert oracle.checks.calc_diff(got, want) <= oracle.checks.CALC_DIFF_MAX


def _dequant(w):
    p = np.pad(w, ((0, -w.shape[0] % 128), (0, -w.shape[1] % 128)))
    q, sf = quantise.quantise_weight(p[None])
    return gemm.dequant_weight(q[0], sf[0])[:w.shape[0]]


def test_shared_expert_is_added_to_the_combine(problem):
    x, logits, w13, w2, shared = problem
    routed, _, _ = oracle.block.moe_block(x, logits, w13, w2, KR)
    alone, _, _ = oracle.block.moe_block(x, np.full_like(logits, -np.inf), w13, w2, KR, shared=shared)
    both, _, _ = oracle.block.moe_block(x, logits, w13, w2, KR, shared=shared)
    f = formats.bf16_bits_to_f64
    want = f(routed) + f(alone)
    assert (np.abs(f(both) - want) <= 2.0 ** -8 * (np.abs(want) + np.abs(f(alone)))).all()
