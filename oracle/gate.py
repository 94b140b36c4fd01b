"""Router choice: top-k expert ids and weights from router logits, in float64.

TEST INFRASTRUCTURE ONLY (see the package docstring).

Definition: an expert is usable if its logit is neither NaN nor -inf (+inf
counts as the largest finite float32).  s = sigmoid(l), or the softmax over the
usable experts.  The choice goes by s + bias, or by l without a bias; an expert
for which that is NaN or -inf is never chosen.  Of G groups of consecutive
experts the ``kept`` of the largest score (largest value, or sum of the two
largest s (+ bias)) take part; the kr largest are chosen in descending order.
Ties go to the lowest index.  Weights are s of the chosen, optionally divided
by their sum, times ``scale``; missing choices are id -1 with weight 0.  A score
that float64 cannot hold is 0 (and the weights divided by a sum of such sigmoid
scores are), except in softmax weights that are divided by their sum: those are
exp(l - l') / sum, l' the largest chosen logit.

Pins: ``tests/test_oracle_gate.py`` (hand-computed rows, a sort-free brute
force, shift invariance of the softmax, masked rows).
"""

import numpy as np

F32_MAX = float(np.finfo(np.float32).max)


def scores(logits, sigmoid):
    """(s, usable) in float64."""
    l = np.asarray(logits, dtype=np.float64)
    usable = ~(np.isnan(l) | np.isneginf(l))
    l = np.where(usable, np.minimum(l, F32_MAX), 0.0)
    if sigmoid:
        with np.errstate(over="ignore"):
            s = 1.0 / (1.0 + np.exp(-l))
    else:
        m = np.max(np.where(usable, l, -np.inf), axis=1, keepdims=True)
        m = np.where(np.isfinite(m), m, 0.0)
        with np.errstate(over="ignore"):
            ex = np.where(usable, np.exp(np.where(usable, l - m, 0.0)), 0.0)
        s = ex / np.maximum(ex.sum(axis=1, keepdims=True), 1e-300)
    return np.where(usable, s, 0.0), usable


def choice_keys(logits, sigmoid, bias):
    s, usable = scores(logits, sigmoid)
    if bias is None:
        key = np.where(usable, np.minimum(np.where(usable, logits, 0.0), F32_MAX), -np.inf)
        value = np.where(usable, s, -np.inf)
    else:
        v = s + np.asarray(bias, dtype=np.float64)
        key = np.where(usable & ~np.isnan(v), v, -np.inf)
        value = key
    return s, key, value


def group_scores(key, value, groups, top2):
    T, E = key.shape
    if not top2:
        return key.reshape(T, groups, E // groups).max(axis=2)
    v = np.sort(value.reshape(T, groups, E // groups), axis=2)
    second = v[:, :, -2] if E > groups else np.full((T, groups), -np.inf)
    return v[:, :, -1] + np.where(np.isneginf(second), 0.0, second)


def _cut(values, kept):
    """Smallest difference of unequal values that decides which ``kept`` of these descending values are taken."""
    if kept >= len(values):
        return np.inf
    last = values[kept - 1]
    lower = [last - v for v in values[kept:] if v < last]
    higher = [v - last for v in values[:kept] if v > last] if values[kept] == last else []
    return min(lower[:1] + higher[-1:], default=np.inf)


def gate(logits, kr, sigmoid=False, bias=None, groups=1, kept=1, top2=False, renormalise=True, scale=1.0):
    """(ids int32 [T, kr], weights float64 [T, kr], margin [T]): margin is the smallest difference, in any
    comparison the choice rests on, of two unequal values (inf where there is none).  Where values tie at the
    place of the last one taken, that is also their difference to the nearest unequal ones, which less precise
    arithmetic could add to the tie."""
    logits = np.asarray(logits, dtype=np.float64)
    T, E = logits.shape
    s, key, value = choice_keys(logits, sigmoid, bias)
    ids = np.full((T, kr), -1, dtype=np.int32)
    w = np.zeros((T, kr))
    margin = np.full(T, np.inf)
    gs = group_scores(key, value, groups, top2)
    for t in range(T):
        order = sorted(range(groups), key=lambda g: (-gs[t, g], g))
        margin[t] = min(margin[t], _cut([gs[t, g] for g in order], kept))
        k = key[t].copy()
        for g in order[kept:]:
            k[g * (E // groups):(g + 1) * (E // groups)] = -np.inf
        ranked = sorted((e for e in range(E) if k[e] > -np.inf), key=lambda e: (-k[e], e))
        for a, b in zip(ranked[:kr], ranked[1:kr]):
            if k[a] > k[b]:
                margin[t] = min(margin[t], k[a] - k[b])
        margin[t] = min(margin[t], _cut([k[e] for e in ranked], kr))
        for r, e in enumerate(ranked[:kr]):
            ids[t, r] = e
            w[t, r] = s[t, e]
        if renormalise and not sigmoid and ranked:
            l = np.minimum(logits[t, ranked[:kr]], F32_MAX)
            w[t, :len(l)] = np.exp(l - l.max())
    if renormalise:
        total = w.sum(axis=1, keepdims=True)
        w = np.where(total > 0, w / np.where(total > 0, total, 1.0), 0.0)
    return ids, w * scale, margin
