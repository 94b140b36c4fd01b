"""Pins of the SwiGLU oracle: closed forms, the odd part of silu, the block quantiser."""

import numpy as np

import oracle


def _bits(x):
    return oracle.formats.bf16_round(np.asarray(x, dtype=np.float64))


def test_closed_forms():
    y = np.zeros((1, 16))
    y[0, :8] = [0, 1, -1, 2, -64, 64, 0.5, -0.5]
    y[0, 8:] = [3, 2, 2, 1, 1, 1, 0, 4]
    h = oracle.swiglu.swiglu(_bits(y))[0]
    e = np.e
    want = [0, 2 * e / (e + 1), -2 / (e + 1), 2 * e ** 2 / (1 + e ** 2), -64 * np.exp(-64.0) / (1 + np.exp(-64.0)),
            64 / (1 + np.exp(-64.0)), 0, -2 / (1 + np.exp(0.5))]
    np.testing.assert_allclose(h, want, rtol=1e-14)


def test_odd_part_is_half_the_argument():
    g = oracle.formats.bf16_bits_to_f64(_bits(np.linspace(-20, 20, 256)))
    one = np.ones(256)
    a = oracle.swiglu.swiglu(_bits(np.concatenate([g, one])[None]))
    b = oracle.swiglu.swiglu(_bits(np.concatenate([-g, one])[None]))
    np.testing.assert_allclose(a - b, g[None], atol=1e-12)


def test_quantises_as_the_activation_quantiser():
    rng = np.random.default_rng(3)
    u = _bits(rng.standard_normal((4, 256)))
    # g = 128: silu(g) = g to float64 accuracy, so h = 2**7 u: the same codes, every exponent 7 higher
    g = np.full((4, 256), 128.0)
    y = np.concatenate([_bits(g), u], axis=1)
    q, sf = oracle.swiglu.swiglu_quantise(y)
    q_ref, sf_ref = oracle.quantise.quantise_act(u)
    assert np.array_equal(q, q_ref)
    assert np.array_equal(sf.astype(int), sf_ref.astype(int) + 7)


def test_short_last_block_is_padded_with_zeros():
    rng = np.random.default_rng(4)
    y = _bits(rng.standard_normal((3, 2 * 136)))
    q, sf = oracle.swiglu.swiglu_quantise(y)
    assert q.shape == (3, 256) and sf.shape == (3, 2)
    assert not q[:, 136:].any()
