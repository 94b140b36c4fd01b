"""A CTA whose loads never come keeps its whole cluster from storing.

With BSF_DEBUG_WITHHOLD_LOADS only the last CTA of a cluster that shares a product's K waits in vain (its waits
are bounded); the others finish, and their sums would hold its unfinished partial."""

import pytest
import torch

from block_scaled_fp8_route_gb300 import ops
from tests.gpu_util import require_gpu

pytestmark = pytest.mark.gpu
WITHHOLD_LOADS = 0x100


# (sizes for which K goes over 8, 4 and 2 CTAs or stays in one, one token chunk and several)
@pytest.mark.parametrize("M,N,K", [(1, 128, 7168), (8, 2048, 7168), (37, 7168, 2048), (64, 4096, 7168), (128, 1024, 1024),
                                   (200, 512, 512), (16, 16384, 256)])
def test_nothing_is_stored(M, N, K):
    dev = require_gpu()
    a, sfa = ops.quantise_act(torch.randn(M, K, device=dev).to(torch.bfloat16))
    b, sfb = ops.prepare_dense_weight(torch.randn(N, K, device=dev).to(torch.bfloat16))
    want = ops.dense_gemm(a, sfa, b, sfb, N)
    torch.cuda.synchronize()
    assert ops.device_error() == 0
    d = torch.full((M, N), 7.0, dtype=torch.bfloat16, device=dev)
    ops.dense_gemm(a, sfa, b, sfb, N, d=d, flags=ops.B_TILED | WITHHOLD_LOADS)
    torch.cuda.synchronize()
    assert ops.device_error() & ops.DEVERR_TIMEOUT
    assert (d == 7.0).all()
    assert torch.equal(ops.dense_gemm(a, sfa, b, sfb, N), want)
    assert ops.device_error() == 0
