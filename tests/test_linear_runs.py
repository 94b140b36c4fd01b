"""No issuer and no run of a split product is without a K-block, whose accumulator the epilogue would add unwritten: the
counts of linear's kernel restated over lengths and splits.  CPU-only."""

import pytest

BLOCK, SEGMENT = 64, 1024


def shares(nkb, split):
    """K-blocks of every run of every issuer of every CTA, and how many K-blocks a run may have."""
    issuers = 2 if nkb // split >= 2 else 1
    most = -(-(-(-nkb // split)) // issuers)
    runs = -(-most * BLOCK // SEGMENT)
    for rank in range(split):
        mine = nkb * (rank + 1) // split - nkb * rank // split
        for me in range(issuers):
            count = (mine - me + issuers - 1) // issuers
            yield runs, [count * (r + 1) // runs - count * r // runs for r in range(runs)]


@pytest.mark.parametrize("split", range(1, 9))
def test_split_products(split):
    for nkb in [n for n in range(1, 1200) if split == 1 or n >= 2 * split] + [4096, 131071, 262144]:
        for runs, of_run in shares(nkb, split):
            assert max(of_run) * BLOCK <= SEGMENT
            assert min(of_run) >= (8 if runs > 1 else 1), (nkb, split, of_run)


def test_pairs():
    for nkb in range(1, 4000):
        for issuers in (1, 2) if nkb > 2 else (1,):
            stages = -(-nkb // issuers)                              # a stage of two issuers' tiles is two K-blocks
            segments = -(-stages * issuers * BLOCK // SEGMENT)
            for i in range(segments):
                n = stages * (i + 1) // segments - stages * i // segments
                assert issuers <= n and n * BLOCK <= SEGMENT // issuers + (BLOCK if segments == 1 else 0)
