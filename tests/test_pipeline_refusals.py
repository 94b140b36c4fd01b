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


M_CAP, K2, N2 = 24, 128, 384


class _Bufs:
    m_cap = M_CAP


@pytest.fixture
def path(monkeypatch):
    def reached(*a, **k):
        raise Reached
    monkeypatch.setattr(MoEPath, "_stage_in", reached)
    p = object.__new__(MoEPath)
    p.E, p.kr, p.T, p.K, p.K2, p.N2, p.bufs, p.two_gemms = E, KR, T, K, K2, N2, _Bufs(), True
    p.z = torch.zeros(T, N2, dtype=BF16)
    return p


IDS, WEIGHTS = torch.zeros(T, KR, dtype=torch.int32), torch.zeros(T, KR)
H2 = torch.zeros(M_CAP, K2, dtype=BF16)


def test_path_takes_what_it_was_made_for(path):
    for h2 in (H2, H2[:M_CAP - 3]):
        with pytest.raises(Reached):
            path.step(X, IDS, WEIGHTS, h2, z=torch.zeros(T, N2, dtype=BF16))
    path.two_gemms = False
    with pytest.raises(Reached):
        path.step(X, IDS, WEIGHTS)


@pytest.mark.parametrize("name,value", [
    ("x", torch.zeros(T + 1, K, dtype=BF16)), ("x", torch.zeros(T, K + 128, dtype=BF16)), ("x", torch.zeros(T, K)),
    ("topk_ids", torch.zeros(T - 1, KR, dtype=torch.int32)), ("topk_ids", torch.zeros(T, KR, dtype=torch.int64)),
    ("topk_ids", torch.zeros(T, KR + 1, dtype=torch.int32)), ("topk_weights", torch.zeros(T, KR - 1)),
    ("topk_weights", torch.zeros(T, KR, dtype=BF16)), ("h2", None), ("h2", torch.zeros(M_CAP + 1, K2, dtype=BF16)),
    ("h2", torch.zeros(M_CAP, K2 - 64, dtype=BF16)), ("h2", torch.zeros(M_CAP, K2)),
    ("z", torch.zeros(T, K, dtype=BF16)), ("z", torch.zeros(T, N2)), ("z", torch.zeros(N2, T, dtype=BF16).t()),
    ("x", X.to("meta")), ("topk_ids", IDS.to("meta")), ("topk_weights", WEIGHTS.to("meta")), ("h2", H2.to("meta"))])
def test_path_refuses_other_inputs(path, name, value):
    args = dict(x=X, topk_ids=IDS, topk_weights=WEIGHTS, h2=H2, z=None)
    args[name] = value
    with pytest.raises(ValueError, match=f"^{name}: "):
        path.step(**args)
