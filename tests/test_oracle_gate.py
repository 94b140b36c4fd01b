"""Pins of the router-choice oracle: hand-computed rows, a sort-free brute force, invariances."""

import math

import numpy as np
import pytest

import oracle


def test_hand_computed_rows():
    l = np.array([[math.log(1), math.log(2), math.log(4), math.log(1)]])
    ids, w, _ = oracle.gate.gate(l, 2, renormalise=False)
    assert ids.tolist() == [[2, 1]]
    np.testing.assert_allclose(w, [[0.5, 0.25]], rtol=1e-14)
    ids, w, _ = oracle.gate.gate(l, 2, renormalise=True, scale=3.0)
    np.testing.assert_allclose(w, [[2.0, 1.0]], rtol=1e-14)
    # sigmoid(0) = 1/2, sigmoid(log 3) = 3/4; the bias moves the choice, never the weight
    l = np.array([[0.0, math.log(3), 0.0, 0.0]])
    ids, w, _ = oracle.gate.gate(l, 2, sigmoid=True, bias=np.array([0, 0, 0, 0.5]), renormalise=False)
    assert ids.tolist() == [[3, 1]]
    np.testing.assert_allclose(w, [[0.5, 0.75]], rtol=1e-14)


def test_groups_by_largest_and_by_two_largest():
    l = np.array([[3.0, -9.0, 2.0, 1.9, 1.0, 0.9]])
    assert oracle.gate.gate(l, 2, groups=3, kept=1)[0].tolist() == [[0, 1]]
    # sigmoid sums: 0.9526 + 0.0001, 0.8808 + 0.8699, 0.7311 + 0.7109
    assert oracle.gate.gate(l, 2, sigmoid=True, groups=3, kept=1, top2=True)[0].tolist() == [[2, 3]]
    assert oracle.gate.gate(l, 2, sigmoid=True, groups=3, kept=2, top2=True)[0].tolist() == [[2, 3]]
    assert oracle.gate.gate(l, 3, sigmoid=True, groups=3, kept=2, top2=True)[0].tolist() == [[2, 3, 4]]


def test_ties_masks_and_nothing_left():
    l = np.array([[1.0, 2.0, 2.0, 2.0], [-np.inf, 0.0, np.nan, -np.inf], [-np.inf] * 4, [np.inf, 1.0, np.inf, 0.0]])
    ids, w, _ = oracle.gate.gate(l, 3)
    assert ids.tolist() == [[1, 2, 3], [1, -1, -1], [-1, -1, -1], [0, 2, 1]]
    np.testing.assert_allclose(w, [[1 / 3] * 3, [1, 0, 0], [0, 0, 0], [0.5, 0.5, 0]], rtol=1e-12)


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("groups,kept,top2", [(1, 1, False), (4, 2, False), (4, 2, True)])
def test_brute_force(sigmoid, groups, kept, top2):
    rng = np.random.default_rng(7)
    l = rng.standard_normal((40, 20))
    b = rng.standard_normal(20) * 0.1
    ids, w, _ = oracle.gate.gate(l, 3, sigmoid=sigmoid, bias=b, groups=groups, kept=kept, top2=top2)
    for t in range(40):
        s = 1 / (1 + np.exp(-l[t])) if sigmoid else np.exp(l[t]) / np.exp(l[t]).sum()
        v = (s + b).reshape(groups, -1)
        gs = [sum(sorted(r)[-2:]) if top2 else max(r) for r in v]
        open_groups = [g for g in range(groups) if sum(gs[o] > gs[g] for o in range(groups)) < kept]
        cand = {e: (s + b)[e] for e in range(20) if e // (20 // groups) in open_groups}
        want = [e for e in cand if sum(x > cand[e] for x in cand.values()) < 3]
        assert set(ids[t]) == set(want)
        np.testing.assert_allclose(w[t], s[ids[t]] / s[ids[t]].sum(), rtol=1e-12)


def test_softmax_weights_do_not_move_with_a_shift():
    rng = np.random.default_rng(8)
    l = rng.standard_normal((10, 33))
    a, b = oracle.gate.gate(l, 4, renormalise=False), oracle.gate.gate(l + 500.0, 4, renormalise=False)
    assert np.array_equal(a[0], b[0])
    np.testing.assert_allclose(a[1], b[1], rtol=1e-11)
