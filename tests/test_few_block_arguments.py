"""A block of few tokens packs no rows and refuses the arguments that say how.  CPU-only."""

import pytest
import torch

from block_scaled_fp8_route_gb300 import MoEBlock, ops
from tests.test_few_tokens_refusals import Reached, no_quantisation  # noqa: F401


def block(**kw):
    w13, w2 = torch.zeros(8, 256, 256, dtype=torch.bfloat16), torch.zeros(8, 256, 128, dtype=torch.bfloat16)
    return MoEBlock(8, 2, 4, 256, 128, w13, w2, device="cpu", **kw)


@pytest.mark.parametrize("kw", [dict(layout=ops.MASKED, align_or_max_m=64), dict(align_or_max_m=64), dict(expected_m=4)])
def test_arguments_of_packed_rows(no_quantisation, kw):  # noqa: F811
    with pytest.raises(ValueError, match="few_tokens: layout"):
        block(few_tokens=True, **kw)
    with pytest.raises(Reached):
        block(**kw)


def test_their_defaults_are_taken(no_quantisation):  # noqa: F811
    with pytest.raises(Reached):
        block(few_tokens=True, layout=ops.CONTIGUOUS, align_or_max_m=128, expected_m=0)
