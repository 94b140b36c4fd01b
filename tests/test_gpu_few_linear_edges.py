"""Calls of few_token_moe and linear that their documentation allows: masked tokens that hold anything, a layer onto its own
input, and operands whose offsets pass 32 bits."""

import numpy as np
import pytest
import torch

import oracle
from block_scaled_fp8_route_gb300 import ops
from tests.gpu_util import require_gpu
from tests.test_gpu_few_tokens import Layer, inputs

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def dev():
    return require_gpu()


@pytest.mark.parametrize("fmt", ["fp8", "bf16"])
def test_masked_tokens_and_choices_may_hold_anything(dev, fmt):
    layer = Layer(dev, 8, 384, 256, fmt=fmt)
    x, ids, p = inputs(dev, 12, 384, 8, 3)
    ids[4], ids[11], ids[7, 1] = -1, -1, -5
    clean = layer.call(x, ids, p)
    layer.check(clean, x, ids, p)
    x[4], x[11] = float("nan"), float("inf")
    p[4], p[11], p[7, 1] = float("nan"), -float("inf"), float("nan")
    z = layer.call(x, ids, p)
    assert ops.device_error() == 0
    assert torch.equal(z, clean) and torch.count_nonzero(z[[4, 11]]) == 0


@pytest.mark.parametrize("fmt", ["fp8", "bf16"])
def test_onto_its_own_input(dev, fmt):
    layer = Layer(dev, 8, 2176, 256, 128, fmt=fmt)
    for T in (1, 9, 32):
        x, ids, p = inputs(dev, T, 2176, 8, 3, T)
        want = layer.call(x, ids, p, addend=x)
        layer.check(want, x, ids, p, addend=x)
        assert layer.call(x, ids, p, addend=x, z=x) is x
        assert torch.equal(x, want)


@pytest.mark.parametrize("out", [BF16, torch.float32])
def test_offsets_past_32_bits(dev, out):
    """Rows of x, of the residual and of y whose elements are more than 2**31 from the first."""
    T, N, K, pitch = (1 << 19) + 37, 72, 64, 4104
    g = torch.Generator(device=dev).manual_seed(1)
    wide = torch.empty(T, pitch, dtype=BF16, device=dev)
    x = wide[:, 8:8 + K]
    x.copy_(torch.randn(T, K, device=dev, generator=g))
    w = torch.randn(N, K, device=dev, generator=g).to(BF16)
    big = torch.empty(T, pitch, dtype=out, device=dev)
    y, r = big[:, :N], big[:, 2000:2000 + N]
    r.copy_(torch.randn(T, N, device=dev, generator=g))
    ops.linear(x, w, activation="relu", residual=r, out=y)
    assert ops.device_error() == 0
    for rows in (slice(0, 40), slice(T // 2, T // 2 + 40), slice(T - 400, T)):
        args = [t[rows].double().cpu().numpy() for t in (x, r)]
        ref = oracle.linear.linear(args[0], w.double().cpu().numpy(), None, "relu", args[1])
        tol = oracle.linear.bound(args[0], w.double().cpu().numpy(), None, "relu", args[1],
                                  eps=2.0 ** -8 if out == BF16 else 2.0 ** -24)
        assert np.all(np.abs(y[rows].double().cpu().numpy() - ref) <= tol)
    # every row, against the library's product of the same values (within both bounds)
    other = torch.relu(x.float() @ w.float().t()) + r.float()
    assert torch.all((y.float() - other).abs() <= 2.0 ** -7 * other.abs() + 1e-3)
