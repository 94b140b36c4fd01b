"""Pins of the float64 product with an epilogue: values by hand, torch's activations, and the bound against a float32
evaluation."""

import numpy as np
import pytest
import torch

from oracle import linear


def test_by_hand():
    x, w = np.array([[1.0, 2.0], [-3.0, 4.0]]), np.array([[5.0, 6.0]])
    assert np.array_equal(linear.linear(x, w, np.array([0.5]), "relu", np.array([[1.0], [2.0]])), [[18.5], [11.5]])
    assert np.array_equal(linear.linear(-x, w, np.array([0.5]), "relu"), [[0.0], [0.0]])


@pytest.mark.parametrize("name,fn", [
    ("relu", torch.relu), ("silu", torch.nn.functional.silu), ("sigmoid", torch.sigmoid),
    ("gelu", torch.nn.functional.gelu), ("gelu_tanh", lambda v: torch.nn.functional.gelu(v, approximate="tanh"))])
def test_activations(name, fn):
    v = torch.linspace(-12, 12, 4801, dtype=torch.float64)
    got = linear.activate(v.numpy(), name)
    assert np.allclose(got, fn(v).numpy(), rtol=1e-11, atol=1e-14)
    slope = np.abs(np.diff(got)).max() / (24 / 4800)
    assert slope <= 1.13                                             # what the bound counts on


def test_a_float32_evaluation_is_within_the_bound():
    r = np.random.default_rng(0)
    x, w, b = (r.standard_normal(s).astype(np.float32).astype(np.float64) for s in ((9, 400), (33, 400), (33,)))
    got = np.float32(x) @ np.float32(w).T + np.float32(b)
    ref, tol = linear.linear(x, w, b), linear.bound(x, w, b)
    assert np.all(np.abs(got - ref) <= tol) and np.median(np.abs(got - ref) / tol) > 1e-4
