"""A single row is taken whatever the stride of the view that it comes from: the same bits as a compact row."""

import pytest
import torch

from block_scaled_fp8_route_gb300 import ops
from tests.gpu_util import require_gpu


@pytest.mark.parametrize("cols", [1, 7, 8, 128, 1001])
@pytest.mark.parametrize("stride", [0, 3, 1001, 1 << 30])
def test_stride_of_a_single_row_stays_in_range(cols, stride):
    t = torch.empty_strided((1, cols), (stride, 1), device="meta")
    ld = ops._row_stride(t, 1, cols, "t")
    assert cols <= ld < cols + 8 and ld % 8 == 0


def test_strides_of_several_rows_are_their_own():
    for ld in (200, 203, 1 << 30):
        assert ops._row_stride(torch.empty_strided((2, 200), (ld, 1), device="meta"), 2, 200, "t") == ld


@pytest.fixture(scope="module")
def dev():
    return require_gpu()


def _strided(row, stride):
    """The same values as a [1, n] view that claims this stride."""
    return torch.as_strided(row, (1, row.shape[1]), (stride, 1))


@pytest.mark.gpu
@pytest.mark.parametrize("stride", [0, 1, 1003, 1 << 25, 1 << 40])
def test_gate(dev, stride):
    for E in (64, 77, 256):
        logits = torch.randn(1, E, device=dev)
        got, want = ops.gate(_strided(logits, stride), 4), ops.gate(logits, 4)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.gpu
@pytest.mark.parametrize("stride", [0, 1, 1003, 1 << 25, 1 << 40])
def test_swiglu(dev, stride):
    y = torch.randn(1, 2 * 136, device=dev).to(torch.bfloat16)
    got, want = ops.swiglu_quantise(_strided(y, stride)), ops.swiglu_quantise(y)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1][:, :1], want[1][:, :1])


@pytest.mark.gpu
@pytest.mark.parametrize("stride", [0, 1, 1003, 1 << 25, 1 << 40])
@pytest.mark.parametrize("N", [256, 205])
def test_dense(dev, stride, N):
    a, sfa = ops.quantise_act(torch.randn(1, 256, device=dev).to(torch.bfloat16))
    b, sfb = ops.prepare_dense_weight(torch.randn(N, 256, device=dev).to(torch.bfloat16))
    c = torch.randn(1, N, device=dev).to(torch.bfloat16)
    want = ops.dense_gemm(a, sfa, b, sfb, N, addend=c)
    out = torch.full((N + 16,), 7.0, dtype=torch.bfloat16, device=dev)
    ops.dense_gemm(a, sfa, b, sfb, N, addend=_strided(c, stride), d=_strided(out[:N].view(1, N), stride))
    assert torch.equal(out[:N].view(1, N), want) and (out[N:] == 7.0).all()
