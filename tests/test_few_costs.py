"""How many costs beyond one the first kernel of few_token_moe may meet: what its packed words have room for.  CPU-only."""

import torch

from tests.few_costs import costs_beyond_one, most_costs


def test_most_costs_of_1024_assignments():
    best = [0] * 1025                                                # of so many assignments, at most 32 an expert
    for n in range(1, 1025):
        best[n] = max(best[n - 1], *(best[n - k] + costs_beyond_one(k) for k in range(1, min(n, 32) + 1)))
    assert best[1024] == 122 < 1 << 11
    assert 32 * costs_beyond_one(32) == 96 < 1 << 8                  # 32 experts of all tokens each


def test_the_routing_reaches_it():
    ids = most_costs(1024, 5, 7)
    assert all(len(set(row.tolist())) == 32 for row in ids)
    counts = torch.bincount(ids.flatten().long(), minlength=1024)
    assert sum(costs_beyond_one(int(n)) for n in counts if n) == 122
