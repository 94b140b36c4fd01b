"""Pins of the router-choice oracle's margin around ties, and of its softmax weights far below the largest logit."""

import numpy as np
import pytest

import oracle


def _logit(s):
    return np.log(s) - np.log1p(-s)


def test_margin_looks_past_a_tie_of_experts():
    # scores .5 .5 .5-1e-9 .25: one of the tied two is taken, and the third is 1e-9 away
    l = _logit(np.array([[0.25, 0.5 - 1e-9, 0.5, 0.5]]))
    bias = np.zeros(4)
    ids, _, margin = oracle.gate.gate(l, 1, sigmoid=True, bias=bias)
    assert ids.tolist() == [[2]]
    np.testing.assert_allclose(margin, 1e-9, rtol=1e-6)
    # both of the tied ones are taken: the nearest other one still decides
    _, _, margin = oracle.gate.gate(l, 2, sigmoid=True, bias=bias)
    np.testing.assert_allclose(margin, 1e-9, rtol=1e-6)
    # a value just above a tie that is cut counts, one above a tie that is taken whole does not
    l = _logit(np.array([[0.5, 0.5, 0.5 + 1e-9, 0.25]]))
    for kr, want in ((2, 1e-9), (3, 1e-9), (4, 1e-9)):     # (the order of the taken rests on it, too)
        np.testing.assert_allclose(oracle.gate.gate(l, kr, sigmoid=True, bias=bias)[2], want, rtol=1e-6)


def test_margin_looks_past_a_tie_of_groups():
    # groups of one: scores 1 (to float64's last bit), 1, 1 - 9e-14
    l = np.array([[30.0, 100.0, 200.0]])
    ids, _, margin = oracle.gate.gate(l, 1, sigmoid=True, groups=3, kept=1, top2=True)
    assert ids.tolist() == [[1]]
    np.testing.assert_allclose(margin, np.exp(-30.0), rtol=1e-2)
    l = _logit(np.array([[0.5, 0.5, 0.5 + 1e-9, 0.25]]))
    for kept, want in ((1, 1e-9), (2, 1e-9), (3, 0.25)):
        margin = oracle.gate.gate(l, 1, sigmoid=True, groups=4, kept=kept, top2=True)[2]
        np.testing.assert_allclose(min(margin[0], 0.25), min(want, _best_gap(l, kept)), rtol=1e-6)


def _best_gap(l, kept):
    """Gap of the two largest logits of the kept groups, by which the one expert is chosen."""
    srt = np.sort(l[0])[::-1][:kept]
    return srt[0] - srt[1] if kept > 1 else np.inf


def test_cut_directly():
    cut = oracle.gate._cut
    assert cut([3.0, 2.0, 1.0], 3) == np.inf
    assert cut([3.0, 2.0, 1.0], 2) == 1.0
    assert cut([3.0, 2.0, 2.0, 0.5], 2) == 1.0             # tie at the cut: 3 - 2 above, 2 - 0.5 below
    assert cut([2.25, 2.0, 2.0, 0.5], 3) == 1.5            # the tie is taken whole
    assert cut([2.0, 2.0, 2.0], 1) == np.inf
    assert cut([1.0, 1.0, -np.inf], 1) == np.inf


@pytest.mark.parametrize("shift", [0.0, -700.0, -800.0, -1e30])
def test_softmax_weights_of_chosen_far_below_the_largest(shift):
    """The bias keeps the largest logit out; the weights are those of the chosen logits alone."""
    l = np.array([[0.0, 1.0, -1.0, 2.0]]) + np.array([[0.0, shift, shift, shift]])
    bias = np.array([-5.0, 3.0, 2.0, 1.0])
    ids, w, _ = oracle.gate.gate(l, 2, bias=bias)
    assert ids.tolist() == [[1, 2]]
    d = np.exp(l[0, [1, 2]] - l[0, [1, 2]].max())
    np.testing.assert_allclose(w[0], d / d.sum(), rtol=1e-12)
