"""GPU parity of the router choice (``gate``) with the float64 oracle.

Ids are equal wherever no comparison of the choice is nearer than 4e-6 (a
float32 score is within 2**-21 = 4.8e-7 of its exact value, a sum of two and a
bias within 1.2e-6); exact ties stay in.  Weights: float32 exp of an argument
that was itself rounded (relative error up to |l - m| 2**-24, doubled for the
function's own 2 ulp), a sum of E terms and a division, so
|w - w64| <= 2**-24 (4 spread + E / 16 + 64) w64 with spread the largest |l - m|
of a usable expert that could matter (at most 104, below which exp is 0), plus
2**-126 below the normal range.
"""

import numpy as np
import pytest
import torch

import oracle
from block_scaled_fp8_route_gb300 import ops
from tests.gpu_util import require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    return require_gpu()


def _check(logits, kr, dev, sigmoid=False, bias=None, groups=1, kept=1, top2=False, renormalise=True, scale=1.0,
           most_unclear=0.02):
    ids, w = ops.gate(logits, kr, score="sigmoid" if sigmoid else "softmax", bias=bias, groups=groups,
                      kept_groups=kept, group_score="top2" if top2 else "max", renormalise=renormalise, scale=scale)
    l64 = logits.double().cpu().numpy()
    b64 = None if bias is None else bias.double().cpu().numpy()
    ids_ref, w_ref, margin = oracle.gate.gate(l64, kr, sigmoid, b64, groups, kept, top2, renormalise, scale)
    clear = margin > 4e-6 if (bias is not None or top2) else np.ones(len(l64), bool)
    assert (~clear).mean() <= most_unclear
    assert np.array_equal(ids.cpu().numpy()[clear], ids_ref[clear])
    assert ids.dtype == torch.int32 and w.dtype == torch.float32
    fin = np.isfinite(l64)
    spread = np.minimum(104.0, np.where(fin, np.abs(l64), 0).max(axis=1, keepdims=True) * (1 if sigmoid else 2))
    tol = 2.0 ** -24 * (4 * spread + l64.shape[1] / 16 + 64)
    err = np.abs(w.double().cpu().numpy() - w_ref)[clear]
    assert (err <= (tol * np.abs(w_ref) + 2.0 ** -126)[clear]).all()
    return ids, w


def _logits(T, E, dtype, dev, seed=0, sd=1.5):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(T, E, generator=g) * sd).to(dtype).to(dev)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,E,kr", [(1, 8, 2), (1, 256, 8), (3, 1, 1), (5, 7, 7), (64, 33, 4), (129, 100, 6),
                                    (257, 160, 6), (1000, 255, 8), (77, 384, 8), (40, 512, 10), (9, 1000, 32),
                                    (6, 1024, 9)])
@pytest.mark.parametrize("sigmoid", [False, True])
def test_choice_by_logit(dev, dtype, T, E, kr, sigmoid):
    _check(_logits(T, E, dtype, dev, seed=T + E), kr, dev, sigmoid=sigmoid, renormalise=True, scale=2.5)
    _check(_logits(T, E, dtype, dev, seed=T + E + 1), kr, dev, sigmoid=sigmoid, renormalise=False)


@pytest.mark.parametrize("E,groups,kept,kr", [(256, 16, 4, 8), (256, 8, 4, 8), (256, 4, 1, 8), (160, 8, 3, 6),
                                              (192, 8, 3, 6), (60, 12, 5, 4), (96, 32, 7, 5), (32, 32, 6, 6),
                                              (1024, 32, 5, 20), (128, 2, 1, 8), (35, 7, 2, 3), (512, 1, 1, 8)])
@pytest.mark.parametrize("top2", [False, True])
@pytest.mark.parametrize("sigmoid,biased", [(True, True), (False, True), (True, False), (False, False)])
def test_groups(dev, E, groups, kept, kr, top2, sigmoid, biased):
    logits = _logits(300, E, torch.float32, dev, seed=E + groups)
    g = torch.Generator().manual_seed(5)
    bias = (torch.randn(E, generator=g) * 0.1).to(dev) if biased else None
    # (softmax scores of 1024 experts are near 1e-3, so more of their comparisons are close)
    _check(logits, kr, dev, sigmoid=sigmoid, bias=bias, groups=groups, kept=kept, top2=top2, renormalise=sigmoid,
           most_unclear=0.25)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("E,groups,kept,kr", [(64, 1, 1, 6), (256, 8, 3, 8), (60, 12, 5, 4)])
def test_renormalised_weights_far_below_the_largest_logit(dev, dtype, E, groups, kept, kr):
    """A bias keeps out the experts of the largest logits, so the chosen scores are all near exp(-100)."""
    logits = _logits(50, E, torch.float32, dev, seed=E)
    logits[:, 1] = 100.0
    bias = torch.linspace(0.5, 1.5, E, device=dev)[torch.randperm(E, generator=torch.Generator().manual_seed(2))]
    bias[1] = -3.0
    _check(logits.to(dtype), kr, dev, bias=bias, groups=groups, kept=kept)


@pytest.mark.parametrize("groups,kept", [(1, 1), (4, 2)])
def test_ties_go_to_the_lowest_index(dev, groups, kept):
    g = torch.Generator().manual_seed(1)
    for dtype in (torch.float32, torch.bfloat16):
        logits = torch.randint(-2, 3, (400, 96), generator=g).to(dtype).to(dev)
        _check(logits, 8, dev, groups=groups, kept=kept)
        _check(logits, 8, dev, sigmoid=True, groups=groups, kept=kept)
    zero = torch.zeros(3, 40, device=dev)
    zero[1, 5] = -0.0                       # the two zeros tie
    ids, w = _check(zero, 4, dev)
    assert ids.tolist() == [[0, 1, 2, 3]] * 3


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("groups,kept,top2", [(1, 1, False), (8, 3, False), (8, 3, True)])
def test_masked_infinite_and_nan_logits(dev, sigmoid, dtype, groups, kept, top2):
    logits = _logits(60, 64, dtype, dev, seed=3)
    g = torch.Generator().manual_seed(9)
    mask = torch.rand(60, 64, generator=g)
    logits[mask.to(dev) < 0.3] = -float("inf")
    logits[(mask.to(dev) > 0.97)] = float("nan")
    logits[0] = -float("inf")                            # nothing left
    logits[1] = float("nan")
    logits[2, :63] = -float("inf")                       # one left
    logits[3, 8:] = -float("inf")                        # one group left
    logits[4] = torch.finfo(dtype).min                   # the type's lowest value is a finite logit: all tie
    logits[5, 7] = float("inf")
    logits[6, 7] = logits[6, 20] = float("inf")
    logits[7] = torch.finfo(dtype).min
    logits[7, 30] = torch.finfo(dtype).max
    ids, w = _check(logits, 6, dev, sigmoid=sigmoid, groups=groups, kept=kept, top2=top2, most_unclear=0.1)
    assert ids[0].tolist() == [-1] * 6 and w[0].tolist() == [0.0] * 6
    assert ids[1].tolist() == [-1] * 6
    assert ids[2].tolist() == [63] + [-1] * 5
    assert torch.isfinite(w).all()


def test_bias_can_shut_an_expert_out_or_force_it(dev):
    logits = _logits(50, 64, torch.float32, dev, seed=4)
    bias = torch.zeros(64)
    bias[[3, 9]] = -float("inf")
    bias[17] = float("nan")
    bias[40] = float("inf")
    ids, w = _check(logits, 5, dev, sigmoid=True, bias=bias.to(dev))
    assert (ids[:, 0] == 40).all()
    for e in (3, 9, 17):
        assert not (ids == e).any()


def test_vanishing_scores(dev):
    """Sigmoid scores that are all zero in float32: ids by logit, weights zero instead of 0 / 0."""
    logits = torch.full((2, 16), -1000.0, device=dev)
    logits[1, 3] = -999.0
    ids, w = ops.gate(logits, 2, score="sigmoid")
    assert ids.tolist() == [[0, 1], [3, 0]] and w.abs().max().item() == 0.0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("off,extra", [(0, 0), (1, 1), (3, 5), (0, 4), (4, 64)])
def test_row_strides_and_offsets(dev, dtype, off, extra):
    for E in (64, 72, 256):
        wide = _logits(37, E + off + extra, dtype, dev, seed=off)
        _check(wide[:, off:off + E], 8, dev)
        _check(wide[:, off:off + E], 8, dev, sigmoid=True, groups=8, kept=3, top2=False)


def test_offsets_past_32_bits(dev):
    """T * ld above 2**31 elements: the last rows are read where they are."""
    T, ld, E = 2100, 1 << 20, 64
    wide = torch.empty(T * ld, dtype=torch.bfloat16, device=dev).view(T, ld)
    tail = _logits(20, E, torch.bfloat16, dev, seed=6)
    view = wide[:, :E]
    view.zero_()
    view[-20:] = tail
    ids, w = ops.gate(view, 4)
    ids_ref, w_ref = ops.gate(tail, 4)
    assert torch.equal(ids[-20:], ids_ref) and torch.equal(w[-20:], w_ref)


def test_empty_batch_and_given_outputs(dev):
    ids, w = ops.gate(torch.empty(0, 16, device=dev), 2)
    assert ids.shape == (0, 2) and w.shape == (0, 2)
    a = torch.full((5, 4), 77, dtype=torch.int32, device=dev)
    b = torch.full((5, 4), 7.0, device=dev)
    out = ops.gate(_logits(4, 16, torch.float32, dev), 4, topk_ids=a[:4], topk_weights=b[:4])
    assert out[0].data_ptr() == a.data_ptr()
    assert (a[4] == 77).all() and (b[4] == 7.0).all() and (a[:4] < 16).all()


def test_other_stream_and_repeat_runs(dev):
    logits = _logits(3000, 256, torch.float32, dev, seed=8)
    kw = dict(score="sigmoid", groups=16, kept_groups=4, group_score="top2")
    ids, w = ops.gate(logits, 8, **kw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        i2, w2 = ops.gate(logits, 8, stream=side, **kw)
        side.synchronize()
        assert torch.equal(ids, i2) and torch.equal(w, w2)
