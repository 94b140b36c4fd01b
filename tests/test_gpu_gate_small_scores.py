"""Scores far below 1 decide a choice with float32's relative accuracy, not with its absolute one.

A sigmoid score is within 7 * 2**-24 of its size (expf 2 units in the last place, 1 + e half of one, the
reciprocal one), a softmax score of an exact l - m within 2**-22, and the sum of two is rounded once more: two
group scores that differ by more than 2 * 8 * 2**-24 = 2**-20 of their size are never mistaken for each other.
The rows below put two groups (or two experts) between that and 2**-18.5 of each other, at logits of -20 to -80."""

import numpy as np
import pytest
import torch

from block_scaled_fp8_route_gb300 import ops
from tests.gpu_util import require_gpu

pytestmark = pytest.mark.gpu
MARGIN = 2.0 ** -20


def _sigmoid(l):
    return 1.0 / (1.0 + np.exp(-l))


def _near_pairs(n, score, seed):
    """(a [n, 2], b [n, 2]) float32: the two largest logits of two groups whose score sums nearly agree."""
    rng = np.random.default_rng(seed)
    x = rng.uniform(-80, -20, 8 * n).astype(np.float32)
    a = np.stack([x, x - np.float32(2)], 1)
    total = score(a.astype(np.float64)).sum(1)
    z = (x + np.float32(0.0963)).astype(np.float32)
    rest = total * (1 + rng.choice([-1, 1], len(x)) * 2.0 ** rng.uniform(-19.9, -18.6, len(x)))
    rest -= score(z.astype(np.float64))
    w = np.log(rest).astype(np.float32)                  # (scores this small are exp(l) but for 1e-9 of them)
    b = np.stack([z, w], 1)
    rel = score(b.astype(np.float64)).sum(1) / total - 1
    keep = (np.abs(rel) > MARGIN * 1.01) & (np.abs(rel) < 2.0 ** -18.5) & (w < z)
    assert keep.sum() >= n
    return a[keep][:n], b[keep][:n], rel[keep][:n]


@pytest.mark.parametrize("E", [64, 256, 20, 384])
@pytest.mark.parametrize("sigmoid", [True, False])
def test_group_scores_of_the_two_largest(E, sigmoid):
    dev = require_gpu()
    n, G = 2000, 4
    per = E // G
    a, b, rel = _near_pairs(n, _sigmoid if sigmoid else np.exp, E)
    rng = np.random.default_rng(E + 1)
    l = np.full((n, G, per), -np.inf, np.float32)
    l[:, 3, 0] = 0.0                                     # the row's largest, in a group of its own; l - m is exact
    order = rng.random((n, per)).argsort(1)              # places in a group
    flip = rng.random(n) < 0.5                           # which of the two groups comes first
    rows = np.arange(n)
    for pair, group in ((a, np.where(flip, 1, 0)), (b, np.where(flip, 0, 1))):
        for i in range(2):
            l[rows, group, order[:, i]] = pair[:, i]
    ids, _ = ops.gate(torch.from_numpy(l.reshape(n, E)).to(dev), 2, score="sigmoid" if sigmoid else "softmax", groups=G,
                      kept_groups=2, group_score="top2", renormalise=False)
    best = np.where(rel > 0, np.where(flip, 0, 1), np.where(flip, 1, 0))
    want = np.stack([np.full(n, 3 * per), best * per + order[:, 0]], 1)
    wrong = (ids.cpu().numpy() != want).any(1)
    assert not wrong.any(), f"{wrong.sum()} of {n} rows"


@pytest.mark.parametrize("E", [40, 256, 512])
@pytest.mark.parametrize("sigmoid", [True, False])
def test_neighbouring_logits_with_a_bias_of_zero(E, sigmoid):
    """Two neighbouring float32 logits have scores 2**-18 and more apart, and the larger one stands behind."""
    dev = require_gpu()
    n = 2000
    rng = np.random.default_rng(E)
    x = rng.uniform(-80, -32.5, n).astype(np.float32)
    l = np.full((n, E), -np.inf, np.float32)
    l[:, 1] = 0.0
    l[:, 5] = x
    l[:, E - 2] = np.nextafter(x, np.float32(0))
    ids, w = ops.gate(torch.from_numpy(l).to(dev), 3, score="sigmoid" if sigmoid else "softmax",
                      bias=torch.zeros(E, device=dev), renormalise=False)
    wrong = (ids.cpu().numpy() != np.array([1, E - 2, 5])).any(1)
    assert not wrong.any(), f"{wrong.sum()} of {n} rows"
    l = l.astype(np.float64)[:, [1, E - 2, 5]]
    s = _sigmoid(l) if sigmoid else np.exp(l) / np.exp(l).sum(1, keepdims=True)
    assert (np.abs(w.double().cpu().numpy() - s) <= MARGIN * s).all()
