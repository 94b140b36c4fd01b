"""gate, swiglu_quantise and dense_gemm refuse operands and streams of other devices than the current one,
on which the library would launch.  CPU-only, with stand-ins for the tensors: a call that is let through
reaches a marker in place of the library."""

import pytest
import torch

from block_scaled_fp8_route_gb300 import _lib, ops


class Reached(Exception):
    pass


class Tensor:
    """What the binding asks of a contiguous CUDA tensor."""
    is_cuda = True

    def __init__(self, *shape, dtype, device=0):
        self._meta = torch.empty(shape, dtype=dtype, device="meta")
        self.dtype, self.shape, self.device = dtype, self._meta.shape, f"cuda:{device}"
        self._index = device

    def get_device(self):
        return self._index

    def __getattr__(self, name):
        if name in ("dim", "stride", "is_contiguous", "numel"):
            return getattr(self._meta, name)
        raise AttributeError(name)

    def data_ptr(self):
        return 256

    def record_stream(self, stream):
        pass


class Stream:
    cuda_stream = 0

    def __init__(self, device):
        self.device_index = device


F32, I32, U8, BF16 = torch.float32, torch.int32, torch.uint8, torch.bfloat16


def _gate(dev, stream=None):
    ops.gate(Tensor(4, 64, dtype=F32, device=dev["logits"]), 2, bias=Tensor(64, dtype=F32, device=dev["bias"]),
             topk_ids=Tensor(4, 2, dtype=I32, device=dev["topk_ids"]),
             topk_weights=Tensor(4, 2, dtype=F32, device=dev["topk_weights"]), stream=stream)


def _swiglu(dev, stream=None):
    ops.swiglu_quantise(Tensor(4, 256, dtype=BF16, device=dev["y"]),
                        rows=(Tensor(4, dtype=I32, device=dev["token_of_row"]),
                              Tensor(1, dtype=I32, device=dev["rows_used"])),
                        q=Tensor(4, 128, dtype=U8, device=dev["q"]), sf=Tensor(1, 4, dtype=I32, device=dev["sf"]),
                        stream=stream)


def _dense(dev, stream=None):
    ops.dense_gemm(Tensor(4, 128, dtype=U8, device=dev["a"]), Tensor(1, 4, dtype=I32, device=dev["sfa"]),
                   Tensor(256, 128, dtype=U8, device=dev["b"]), Tensor(1, 256, dtype=I32, device=dev["sfb"]),
                   addend=Tensor(4, 256, dtype=BF16, device=dev["addend"]),
                   d=Tensor(4, 256, dtype=BF16, device=dev["d"]), stream=stream)


OPERANDS = {_gate: ("logits", "bias", "topk_ids", "topk_weights"),
            _swiglu: ("y", "token_of_row", "rows_used", "q", "sf"), _dense: ("a", "sfa", "b", "sfb", "addend", "d")}


@pytest.fixture(autouse=True)
def library(monkeypatch):
    def reached():
        raise Reached
    monkeypatch.setattr(_lib, "load", reached)
    monkeypatch.setattr(ops, "_current_device", lambda: 0, raising=False)


@pytest.mark.parametrize("call", OPERANDS)
def test_all_on_the_current_device(call):
    for stream in (None, Stream(0)):
        with pytest.raises(Reached):
            call(dict.fromkeys(OPERANDS[call], 0), stream)


@pytest.mark.parametrize("call", OPERANDS)
def test_all_on_another_device(call):
    with pytest.raises(ValueError, match="current device cuda:0"):
        call(dict.fromkeys(OPERANDS[call], 1))


@pytest.mark.parametrize("call,name", [(call, name) for call in OPERANDS for name in OPERANDS[call]])
def test_one_on_another_device(call, name):
    devices = dict.fromkeys(OPERANDS[call], 0)
    devices[name] = 1
    with pytest.raises(ValueError, match=f"{name} on cuda:1"):
        call(devices)


@pytest.mark.parametrize("call", OPERANDS)
def test_a_stream_of_another_device(call):
    with pytest.raises(ValueError, match="stream on cuda:1"):
        call(dict.fromkeys(OPERANDS[call], 0), Stream(1))
