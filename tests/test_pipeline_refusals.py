"""MoEBlock refuses, on the host, inputs that its kernels would misread or write past.

CPU-only: the block is a stand-in without weights, and a check that let an argument through would reach
the first library call, which is replaced by a marker."""

import pytest
import torch

from block_scaled_fp8_route_gb300 import MoEBlock, ops
from block_scaled_fp8_route_gb300.pipeline import MoEPath

T, K, E, KR = 6, 256, 8, 2
BF16 = torch.bfloat16


class Reached(Exception):
    pass


@pytest.fixture
def block(monkeypatch):
    def reached(*a, **k):
        raise Reached
    monkeypatch.setattr(ops, "gate", reached)
    path = object.__new__(MoEPath)
    path.E, path.kr, path.T, path.K, path.bufs = E, KR, T, K, None
    path.z = torch.zeros(T, K, dtype=BF16)
    b = object.__new__(MoEBlock)
    b.T, b.K, b.kr, b.gate_args, b.path, b.z, b.shared = T, K, KR, {}, path, path.z, None
    b.topk_ids = torch.zeros(T, KR, dtype=torch.int32)
    b.topk_weights = torch.zeros(T, KR)
    return b


X, LOGITS = torch.zeros(T, K, dtype=BF16), torch.zeros(T, E)


@pytest.mark.parametrize("logits", [LOGITS, LOGITS.to(BF16)])
def test_block_takes_what_it_was_made_for(block, logits):
    with pytest.raises(Reached):
        block.step(X, logits)
    with pytest.raises(Reached):
        block.step(X, logits, z=torch.zeros(T, K, dtype=BF16))


@pytest.mark.parametrize("x", [torch.zeros(T + 1, K, dtype=BF16), torch.zeros(T - 1, K, dtype=BF16),
                               torch.zeros(T, K + 128, dtype=BF16), torch.zeros(T, K // 2, dtype=BF16),
                               torch.zeros(T, K), torch.zeros(T, K, dtype=torch.float16),
                               torch.zeros(T * K, dtype=BF16), torch.zeros(T, K, dtype=BF16, device="meta")])
def test_block_refuses_other_tokens(block, x):
    with pytest.raises(ValueError, match="^x: "):
        block.step(x, LOGITS)


@pytest.mark.parametrize("logits", [torch.zeros(T, E + 1), torch.zeros(T, E - 1), torch.zeros(T + 1, E),
                                    torch.zeros(E), torch.zeros(T, E, dtype=torch.float16),
                                    torch.zeros(T, E, dtype=torch.float64), torch.zeros(T, E, device="meta")])
def test_block_refuses_other_logits(block, logits):
    with pytest.raises(ValueError, match="^logits: "):
        block.step(X, logits)


@pytest.mark.parametrize("z", [torch.zeros(T - 1, K, dtype=BF16), torch.zeros(T, K - 128, dtype=BF16),
                               torch.zeros(T, K), torch.zeros(K, T, dtype=BF16).t(),
                               torch.zeros(T, K, dtype=BF16, device="meta")])
def test_block_refuses_other_outputs(block, z):
    with pytest.raises(ValueError, match="^z: "):
        block.step(X, LOGITS, z=z)
