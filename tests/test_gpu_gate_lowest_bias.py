"""Biases of the type's lowest finite value leave an expert choosable, after every other one.

Such a key is the lowest float32 itself, and a group score of two of them is below float32's range; the
group is still one that can be kept.  Inputs are built so that the choice does not hang on rounding: keys of
unmasked experts are their scores (bias 0), more than 2**-20 apart in a row."""

import numpy as np
import pytest
import torch

import oracle
from block_scaled_fp8_route_gb300 import ops
from tests.gpu_util import require_gpu

pytestmark = pytest.mark.gpu
LOWEST = torch.finfo(torch.float32).min


@pytest.mark.parametrize("E,groups", [(64, 8), (256, 16), (60, 12), (35, 7), (384, 8)])
@pytest.mark.parametrize("top2", [False, True])
@pytest.mark.parametrize("sigmoid", [False, True])
def test_groups_of_lowest_biases_can_be_kept(E, groups, top2, sigmoid):
    dev = require_gpu()
    per = E // groups
    g = torch.Generator().manual_seed(E)
    order = torch.stack([torch.randperm(E, generator=g) for _ in range(40)])
    # sigmoid scores evenly spread in [0.25, 0.75]; softmax scores of evenly spread probabilities
    u = (order + 1).double() / (E + 1)
    logits = (torch.log((0.25 + 0.5 * u) / (0.75 - 0.5 * u)) if sigmoid else torch.log(0.5 + u)).float()
    bias = torch.zeros(E)
    bias[per:] = LOWEST                                  # one group is left whole, the others are lowest
    bias[per + 1] = 0.0                                  # but for one expert of the second
    kept, kr = 3, min(2 * per + 1, 32)
    ids, w = ops.gate(logits.to(dev), kr, score="sigmoid" if sigmoid else "softmax", bias=bias.to(dev), groups=groups,
                      kept_groups=kept, group_score="top2" if top2 else "max")
    ids = ids.cpu().numpy()
    # every key of a lowest bias is the same float32, in the oracle's 64 bits too (LOWEST + s rounds to it)
    s, _ = oracle.gate.scores(logits.double().numpy(), sigmoid)
    key = s + bias.double().numpy()
    assert (key[:, bias.numpy() == LOWEST] == LOWEST).all()
    ids_ref, w_ref, margin = oracle.gate.gate(logits.double().numpy(), kr, sigmoid, bias.double().numpy(), groups,
                                              kept, top2)
    assert (margin > 2.0 ** -20).all()
    assert (ids_ref >= 0).all()
    assert np.array_equal(ids, ids_ref)
    np.testing.assert_allclose(w.cpu().numpy(), w_ref, rtol=1e-5)


def test_every_bias_lowest():
    dev = require_gpu()
    bias = torch.full((64,), LOWEST, device=dev)
    ids, w = ops.gate(torch.zeros(2, 64, device=dev), 6, score="sigmoid", bias=bias, groups=8, kept_groups=2,
                      group_score="top2")
    assert ids.tolist() == [[0, 1, 2, 3, 4, 5]] * 2
    np.testing.assert_allclose(w.cpu().numpy(), 1 / 6, rtol=1e-6)


def test_lowest_and_infinite_biases_in_order():
    """Groups: two lowest, one lowest and one shut out, both shut out, two of the largest finite value."""
    dev = require_gpu()
    inf = float("inf")
    bias = torch.tensor([LOWEST, LOWEST, LOWEST, -inf, -inf, -inf, -LOWEST, -LOWEST], device=dev)
    for kept, want in ((1, [6, 7, -1, -1]), (2, [6, 7, 2, -1]), (3, [6, 7, 0, 1])):
        kr = min(4, 2 * kept)
        ids, _ = ops.gate(torch.zeros(1, 8, device=dev), kr, score="sigmoid", bias=bias, groups=4, kept_groups=kept,
                          group_score="top2")
        assert ids.tolist() == [want[:kr]]
