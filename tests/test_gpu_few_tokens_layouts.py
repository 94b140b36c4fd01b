"""bf16 rows given to few_token_moe as they are, without a word on their layout."""

import pytest
import torch

from block_scaled_fp8_route_gb300 import ops
from tests.gpu_util import require_gpu
from tests.test_gpu_few_tokens import Layer, inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("S", [0, 128])
def test_bf16_rows_with_the_default_flags(S):
    dev = require_gpu()
    layer = Layer(dev, 6, 384, 256, S, fmt="bf16", tiled=False)
    x, ids, p = inputs(dev, 9, 384, 6, 3)
    z = ops.few_token_moe(x, ids, p, layer.w13, None, layer.w2, None, shared=layer.shared)
    layer.check(z, x, ids, p)
    assert torch.equal(z, layer.call(x, ids, p))
