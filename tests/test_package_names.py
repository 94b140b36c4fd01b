"""The operators of the blocks are names of the package, too.  CPU-only."""

import pytest

import block_scaled_fp8_route_gb300 as package


@pytest.mark.parametrize("name", ["gate", "swiglu_quantise", "dense_gemm", "few_token_moe", "few_token_moe_workspace", "linear",
                                  "linear_form"])
def test_names(name):
    assert getattr(package, name) is getattr(package.ops, name)
