"""Both ways to the quotient g / (1 + exp(-g)) of ``swiglu_quantise`` give the same codes.

A lane works on 16 values at once and divides where one of its gates is above 80 in magnitude or not finite;
otherwise it corrects a product with the reciprocal.  So the same gate and up give the same code whatever
their 15 neighbours are."""

import numpy as np
import pytest
import torch

from block_scaled_fp8_route_gb300 import ops
from tests.gpu_util import require_gpu, u8

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    return require_gpu()


def _bf16(bits):
    return torch.from_numpy(np.asarray(bits, dtype=np.uint16).view(np.int16)).view(torch.bfloat16)


def _codes(gate, up, neighbour, dev):
    """Codes and scales of rows of 16-value pieces, 8 of gate and up and 8 whose product is +0."""
    rows, pieces = gate.shape[0], gate.shape[1] // 8
    g = torch.full((rows, pieces, 16), neighbour, dtype=torch.bfloat16)
    u = torch.zeros(rows, pieces, 16, dtype=torch.bfloat16)
    g[:, :, :8], u[:, :, :8] = gate.view(rows, pieces, 8), up.view(rows, pieces, 8)
    y = torch.cat([g.view(rows, -1), u.view(rows, -1)], dim=1)
    q, sf = ops.swiglu_quantise(y.to(dev))
    return q, sf[:, :rows]


def test_every_finite_gate(dev):
    """128 ups (all the bf16 in [1, 2)) for each of 65280 gates.  A last bit that differs shows in the codes where a
    product lies that near to the middle of two codes: of 8.4 million products, about 20."""
    bits = np.concatenate([np.arange(0x0000, 0x7F80), np.arange(0x8000, 0xFF80)])
    gate = _bf16(bits)[:, None].expand(-1, 128).contiguous()
    up = (1 + torch.arange(128) / 128).to(torch.bfloat16).expand(len(bits), 128).contiguous()
    q1, sf1 = _codes(gate, up, 1.0, dev)
    q2, sf2 = _codes(gate, up, 128.0, dev)
    assert torch.equal(sf1, sf2)
    differ = (q1 != q2).any(dim=1).cpu().numpy()
    assert not differ.any(), [hex(b) for b in bits[differ][:8]]


@pytest.mark.parametrize("neighbour", [1.0, 80.0, 128.0, -1.0, -80.0, -100.0])
def test_signs_of_zero(dev, neighbour):
    """Zero gates and ups of either sign beside non-zero ones: the sign of the product, as IEEE arithmetic has it."""
    g = np.array([0.0, -0.0, 0.0, -0.0, 1.0, -1.0, 0.0, -0.0], np.float32)
    u = np.array([1.0, 1.0, -1.0, -1.0, -0.0, -0.0, 0.0, 0.0], np.float32)
    want = (g / (1 + np.exp(-g)) * u).astype(np.float32)
    assert not want.any()
    gate, up = (torch.from_numpy(np.tile(t, 8)).to(torch.bfloat16)[None] for t in (g, u))
    q, _ = _codes(gate, up, neighbour, dev)
    got = u8(q).reshape(8, 16)[:, :8]
    assert np.array_equal(got, np.broadcast_to(np.where(np.signbit(want), 0x80, 0), got.shape))
