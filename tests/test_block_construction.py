"""MoEBlock refuses weights of other types or sizes and arguments that its gate would refuse, before it
quantises anything."""

import pytest
import torch

from block_scaled_fp8_route_gb300 import MoEBlock, MoEPath, ops
from tests.gpu_util import require_gpu

E, KR, T, K, I, S = 8, 2, 4, 256, 128, 64
BF16 = torch.bfloat16


def _weights(K=K, I=I, S=S, dtype=BF16):
    return (torch.zeros(E, 2 * I, K, dtype=dtype), torch.zeros(E, K, I, dtype=dtype),
            (torch.zeros(2 * S, K, dtype=dtype), torch.zeros(K, S, dtype=dtype)))


class Quantised(Exception):
    pass


@pytest.fixture(autouse=True)
def no_quantisation(monkeypatch):
    def quantised(*a, **k):
        raise Quantised
    monkeypatch.setattr(MoEPath, "__init__", quantised)


@pytest.fixture
def no_gate(monkeypatch):
    monkeypatch.setattr(ops, "gate", lambda *a, **k: None)


def _block(w, shared=None, K=K, I=I, device="cpu", **gate):
    return MoEBlock(E, KR, T, K, I, w[0], w[1], shared=shared, device=device, **gate)


def test_matching_weights_are_taken(no_gate):
    for w in (_weights(), _weights(S=8)):
        with pytest.raises(Quantised):
            _block(w, w[2], score="sigmoid", scale=2.0)


def test_weight_types_and_sizes(no_gate):
    w = _weights()
    for dtype in (torch.float32, torch.float16, torch.uint8):
        with pytest.raises(ValueError, match="bfloat16"):
            _block(_weights(dtype=dtype))
        with pytest.raises(ValueError, match="bfloat16"):
            _block(w, _weights(dtype=dtype)[2])
    with pytest.raises(ValueError, match="multiples of 128"):
        _block(_weights(I=72), I=72)
    with pytest.raises(ValueError, match="multiples of 128"):
        _block(_weights(K=200), K=200)
    for shared in (_weights(S=12)[2], _weights(S=0)[2], _weights(K=128)[2], (w[2][0], w[2][1][:, :32]),
                   (w[2][0][0], w[2][1])):
        with pytest.raises(ValueError, match="shared"):
            _block(w, shared)


def test_arguments_that_do_not_say_how_to_choose(no_gate):
    for name in ("stream", "topk_ids", "topk_weights", "logits"):
        with pytest.raises(TypeError, match=name):
            _block(_weights(), **{name: None})


@pytest.mark.gpu
def test_gate_arguments():
    dev = require_gpu()
    w = _weights()
    with pytest.raises(Quantised):
        _block(w, device=dev, score="sigmoid", groups=4, kept_groups=2, bias=torch.zeros(E, device=dev))
    with pytest.raises(ValueError, match="softmax or sigmoid"):
        _block(w, device=dev, score="relu")
    with pytest.raises(ValueError, match="bias"):
        _block(w, device=dev, bias=torch.zeros(E + 1, device=dev))
    with pytest.raises(ValueError, match="bias"):
        _block(w, device=dev, bias=torch.zeros(E))
    for bad in (dict(groups=3), dict(groups=4, kept_groups=5), dict(groups=8, kept_groups=1), dict(scale=float("nan"))):
        with pytest.raises(RuntimeError, match="gate"):
            _block(w, device=dev, **bad)
