"""prepare_dense_weight refuses what it would read as bf16 without being so, before any device call."""

import pytest
import torch

from block_scaled_fp8_route_gb300 import ops


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.uint8, torch.float64])
def test_other_types(dtype):
    with pytest.raises(ValueError, match="^w: expected torch.bfloat16"):
        ops.prepare_dense_weight(torch.zeros(128, 128, dtype=dtype))
    with pytest.raises(ValueError, match="^w: expected torch.bfloat16"):
        ops.prepare_dense_weight(torch.zeros(100, 72, dtype=dtype, device="meta"))


def test_host_weights_and_other_dimensions():
    with pytest.raises(ValueError, match="^w: expected a CUDA tensor"):
        ops.prepare_dense_weight(torch.zeros(128, 128, dtype=torch.bfloat16))
    for shape in ((128,), (1, 128, 128)):
        with pytest.raises(ValueError, match="^w: expected a 2-D tensor"):
            ops.prepare_dense_weight(torch.zeros(shape, dtype=torch.bfloat16))
