"""gate, swiglu_quantise and dense_gemm on a stream that is not the current one: their new outputs do not
take memory whose last use on the current stream may not have run yet, and every operand's memory is kept
until the given stream is done with it, even where the caller drops it right after the call."""

import pytest
import torch

from block_scaled_fp8_route_gb300 import ops
from tests.gpu_util import require_gpu

pytestmark = pytest.mark.gpu
T, E, K, N = 256, 64, 512, 256


@pytest.fixture(scope="module")
def dev():
    return require_gpu()


def _gate(dev):
    logits, bias = torch.randn(T, E, device=dev), torch.randn(E, device=dev)
    return [logits, bias], lambda s, t: ops.gate(t[0], 4, score="sigmoid", bias=t[1], stream=s)


def _swiglu(dev):
    y = torch.randn(T, 2 * K, device=dev).to(torch.bfloat16)
    token = torch.arange(T, dtype=torch.int32, device=dev)
    used = torch.tensor([T], dtype=torch.int32, device=dev)
    return [y, token, used], lambda s, t: ops.swiglu_quantise(t[0], rows=(t[1], t[2]), stream=s)


def _dense(dev):
    a, sfa = ops.quantise_act(torch.randn(T, K, device=dev).to(torch.bfloat16))
    b, sfb = ops.prepare_dense_weight(torch.randn(N, K, device=dev).to(torch.bfloat16))
    c = torch.randn(T, N, device=dev).to(torch.bfloat16)
    return [a, sfa, b, sfb, c], lambda s, t: (ops.dense_gemm(t[0], t[1], t[2], t[3], N, addend=t[4], stream=s),)


@pytest.mark.parametrize("make", [_gate, _swiglu, _dense])
def test_outputs_do_not_reuse_memory_of_pending_work(dev, make):
    tensors, call = make(dev)
    sizes = [(t.shape, t.dtype) for t in call(None, tensors)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    side.wait_stream(torch.cuda.current_stream())
    # blocks of the outputs' sizes whose last use is still to run on the current stream
    torch.cuda._sleep(20_000_000)
    freed = []
    for shape, dtype in sizes:
        t = torch.zeros(shape, dtype=dtype, device=dev)
        freed.append(t.data_ptr())
        del t
    outputs = call(side, tensors)
    assert not {t.data_ptr() for t in outputs} & set(freed)
    torch.cuda.synchronize()
    for got, want in zip(outputs, call(None, tensors)):
        assert torch.equal(got, want)


@pytest.mark.parametrize("make", [_gate, _swiglu, _dense])
def test_operands_outlive_the_call(dev, make):
    tensors, call = make(dev)
    want = call(None, tensors)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)              # the call's kernel waits behind this
    copies = [t.clone() for t in tensors]
    side.wait_stream(torch.cuda.current_stream())
    got = call(side, copies)
    shapes = [(t.shape, t.dtype) for t in copies]
    where = {t.data_ptr() for t in copies}
    del copies
    for shape, dtype in shapes:                    # the same sizes again, on the current stream
        t = torch.zeros(shape, dtype=dtype, device=dev)
        assert t.data_ptr() not in where
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert torch.equal(g, w)
