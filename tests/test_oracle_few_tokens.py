"""Pins of the float64 layer for few tokens: rational arithmetic where the activation is linear, the whole-block
oracle's structure, and the bound against a float32 evaluation with the operands split as the definition says."""

import numpy as np

import oracle
from oracle import few_tokens


def _layer(E=4, K=256, I=128, T=5, kr=2, seed=0):
    r = np.random.default_rng(seed)
    ids = np.stack([r.permutation(E)[:kr] for _ in range(T)])
    return (r.standard_normal((T, K)), ids, r.random((T, kr)), r.standard_normal((E, 2 * I, K)) * 0.05,
            r.standard_normal((E, K, I)) * 0.05)


def test_one_expert_by_hand():
    # K = I = 1: g = 2 * 3, u = 5 * 3, h = g u / (1 + exp(-g)), z = p * 7 h + c
    x, w13, w2 = np.array([[3.0]]), np.array([[[2.0], [5.0]]]), np.array([[[7.0]]])
    z = few_tokens.few_token_moe(x, np.array([[0]]), np.array([[0.5]]), w13, w2, addend=np.array([[11.0]]))
    assert np.isclose(z[0, 0], 0.5 * 7 * (6 * 15 / (1 + np.exp(-6.0))) + 11, rtol=1e-15)


def test_weights_scale_and_add_up():
    x, ids, p, w13, w2 = _layer()
    z = few_tokens.few_token_moe(x, ids, p, w13, w2)
    assert np.allclose(few_tokens.few_token_moe(x, ids, 2 * p, w13, w2), 2 * z, rtol=1e-13)
    twice = np.concatenate([ids, ids], 1)
    assert np.allclose(few_tokens.few_token_moe(x, twice, np.concatenate([p, p], 1), w13, w2), 2 * z, rtol=1e-13)
    none = np.full_like(ids, -1)
    none[:, 0] = 4
    assert not few_tokens.few_token_moe(x, none, p, w13, w2).any()


def test_shared_expert_is_an_expert_with_weight_one():
    x, ids, p, w13, w2 = _layer()
    with_shared = few_tokens.few_token_moe(x, ids, p, w13, w2, shared=(w13[3], w2[3]))
    ones = np.concatenate([ids, np.full((5, 1), 3)], 1), np.concatenate([p, np.ones((5, 1))], 1)
    assert np.allclose(with_shared, few_tokens.few_token_moe(x, *ones, w13, w2), rtol=1e-12)


def _split(v):
    """hi + lo / 16 in E4M3 over blocks of 128, as values."""
    blocks = v.reshape(-1, 128)
    e = np.ceil(np.log2(np.maximum(np.abs(blocks).max(1, keepdims=True), 1e-30) / 448))
    s = blocks / 2.0 ** e
    def code(a):
        return oracle.formats.e4m3_decode(oracle.formats.e4m3_encode(a))
    hi = code(s)
    return ((hi + code((s - hi) * 16) / 16) * 2.0 ** e).reshape(v.shape)


def test_split_of_bf16_values_is_exact_and_of_others_bounded():
    r = np.random.default_rng(1)
    v = oracle.formats.bf16_bits_to_f64(oracle.formats.bf16_round(r.standard_normal((64, 128))))
    top = np.abs(v).max(1, keepdims=True)
    far = np.abs(v) >= top * 2.0 ** -14
    assert np.array_equal(_split(v)[far], v[far])
    # (the low term's quantum is 2**-9 / 16 where the block's largest is scaled to more than 224: 2**-14 / 224 < 2**-21)
    assert np.all(np.abs(_split(v) - v) <= 2.0 ** -21 * top)
    w = r.standard_normal((256, 128)) * np.exp2(r.integers(-30, 1, (256, 128)))
    top = np.abs(w).max(1, keepdims=True)
    assert np.all(np.abs(_split(w) - w) <= np.maximum(2.0 ** -9 * np.abs(w), 2.0 ** -21 * top))


def test_a_float32_evaluation_is_within_the_bound():
    x, ids, p, w13, w2 = _layer(T=8)
    p = p.astype(np.float32)
    ref, tol = few_tokens.few_token_moe(x, ids, p, w13, w2), few_tokens.bound(x, ids, p, w13, w2)
    got = np.zeros_like(ref, dtype=np.float32)
    xs = _split(x).astype(np.float32)
    for t in range(8):
        for e, q in zip(ids[t], p[t]):
            y = w13[e].astype(np.float32) @ xs[t]
            h = _split((q * y[:128] / (1 + np.exp(-y[:128])) * y[128:]).astype(np.float64)).astype(np.float32)
            got[t] += w2[e].astype(np.float32) @ h
    # (x is not bf16 here: its own split adds 2**-9 of every value, which the bound of a bf16 x leaves out)
    exact_x = few_tokens.few_token_moe(_split(x), ids, p, w13, w2)
    assert np.all(np.abs(got - exact_x) <= tol)
    assert np.median(np.abs(got - exact_x) / tol) > 1e-3             # and the bound is not idle
    assert np.all(np.abs(ref) < 1e3)
