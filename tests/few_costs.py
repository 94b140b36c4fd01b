"""The routing of 32 tokens x 32 choices in which experts cost the most beyond one (their tokens in groups of eight)."""

import torch


def costs_beyond_one(tokens):
    return (tokens + 7) // 8 - 1


def most_costs(E, start=0, step=1):
    """ids [32, 32]: 40 experts of 25 tokens and one of 24, experts start, start + step, ...  Assignment s goes to token
    s % 32 and the (s // 25)-th expert, so that an expert's run of 25 names no token twice."""
    s = torch.arange(1024)
    ids = torch.empty(32, 32, dtype=torch.int32)
    ids[s % 32, s // 32] = (start + step * (s // 25)).int() % E
    return ids
