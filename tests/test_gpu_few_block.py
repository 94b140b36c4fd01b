"""MoEBlock with a router of its own and in the form for few tokens: each stage against the oracle on the stage before
it as the GPU left it, the graph against the eager step, and both forms of the block against one another."""

import numpy as np
import pytest
import torch

import oracle
from block_scaled_fp8_route_gb300 import MoEBlock, ops
from tests.gpu_util import bits16, require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    return require_gpu()


def f64(t):
    return oracle.formats.bf16_bits_to_f64(bits16(t))


def dequantised(w):
    """E4M3 weights with 128 x 128 scales in float64, from the oracle's own quantisation; [n, N, K] or [N, K]."""
    if w.dim() == 2:
        pad = torch.nn.functional.pad(w, (0, -w.shape[1] % 128, 0, -w.shape[0] % 128))
        return dequantised(pad[None])[0][:w.shape[0], :w.shape[1]]
    q, sf = oracle.quantise.quantise_weight(bits16(w))
    return np.stack([oracle.gemm.dequant_weight(q[e], sf[e]) for e in range(w.shape[0])])


def problem(T, E=16, K=384, I=256, S=0, seed=0):
    g = torch.Generator().manual_seed(seed)
    bf16 = lambda *shape, s=0.05: (torch.randn(*shape, generator=g) * s).to(torch.bfloat16)  # noqa: E731
    shared = (bf16(2 * S, K), bf16(K, S)) if S else None
    return (bf16(E, 2 * I, K), bf16(E, K, I), shared, bf16(E, K, s=0.2), torch.randn(E, generator=g) * 0.1,
            bf16(T, K, s=1.0), bf16(T, K, s=1.0))


@pytest.mark.parametrize("T", [1, 5, 16, 32])
@pytest.mark.parametrize("S", [0, 128, 72])
def test_stages(dev, T, S):
    E, kr, K, I = 16, 3, 384, 256
    w13, w2, shared, router, bias, x, addend = problem(T, E, K, I, S, T)
    block = MoEBlock(E, kr, T, K, I, w13, w2, shared=shared, device=dev, score="sigmoid", scale=2.5, few_tokens=True,
                     router=(router, bias))
    xd, ad = x.to(dev), addend.to(dev)
    z = block.step(xd, addend=ad).clone()
    assert ops.device_error() == 0

    args = (f64(x), f64(router), bias.double().numpy())
    ref, tol = oracle.linear.linear(*args), oracle.linear.bound(*args)
    assert np.all(np.abs(block.logits.cpu().numpy() - ref) <= tol)
    logits = block.logits.cpu().numpy()
    ids, weights, margin = oracle.gate.gate(logits, kr, sigmoid=True, scale=2.5)
    assert np.array_equal(block.topk_ids.cpu().numpy(), ids)
    np.testing.assert_allclose(block.topk_weights.cpu().numpy(), weights, rtol=2e-6)

    wide_shared = None
    if S:
        # the block quantises gate and up rows apart, each padded to a multiple of 128
        s13 = np.concatenate([dequantised(shared[0][:S]), dequantised(shared[0][S:])])
        wide_shared = (s13, dequantised(shared[1]))
    args = (f64(x), ids, block.topk_weights.cpu().numpy(), dequantised(w13), dequantised(w2), wide_shared, f64(addend))
    ref = oracle.few_tokens.few_token_moe(*args)
    if S % 128:                                                      # (the bound counts blocks of 128)
        pad = lambda w: np.pad(w, ((0, -w.shape[0] % 128), (0, 0)))  # noqa: E731
        wide = (np.concatenate([pad(wide_shared[0][:S]), pad(wide_shared[0][S:])]), np.pad(wide_shared[1], ((0, 0), (0, -S % 128))))
        args = args[:5] + (wide, args[6])
    tol = oracle.few_tokens.bound(*args)
    assert np.all(np.abs(f64(z) - ref) <= tol + 2.0 ** -8 * (np.abs(ref) + tol))

    block.capture(xd, addend=ad)
    block.z.zero_()
    assert torch.equal(block.replay(), z)
    xd.copy_(xd.flip(0))
    ad.copy_(ad.flip(0))
    assert torch.equal(block.replay(), block.step(xd, addend=ad, z=torch.empty_like(z)))


@pytest.mark.parametrize("T", [3, 32])
def test_both_forms_agree_within_fp8(dev, T):
    E, kr, K, I, S = 16, 4, 384, 256, 128
    w13, w2, shared, router, bias, x, _ = problem(T, E, K, I, S, T + 50)
    args = dict(shared=shared, device=dev, score="softmax", router=router)
    few = MoEBlock(E, kr, T, K, I, w13, w2, few_tokens=True, **args)
    chain = MoEBlock(E, kr, T, K, I, w13, w2, **args)
    a, b = few.step(x.to(dev)), chain.step(x.to(dev))
    assert torch.equal(few.topk_ids, chain.topk_ids) and torch.equal(few.logits, chain.logits)
    # the chain rounds x and h to E4M3 (2**-4 of each value at most, a fifth of that on average): within 2e-3
    assert oracle.checks.calc_diff(f64(b), f64(a)) <= 2e-3
    given = few.step(x.to(dev), few.logits.clone(), z=torch.empty_like(a))
    assert torch.equal(given, few.step(x.to(dev)))


def test_masked_tokens_get_the_shared_expert_alone(dev):
    E, kr, K, I, S, T = 16, 2, 384, 256, 256, 6
    w13, w2, shared, _, _, x, _ = problem(T, E, K, I, S, 3)
    block = MoEBlock(E, kr, T, K, I, w13, w2, shared=shared, device=dev, few_tokens=True)
    logits = torch.randn(T, E, device=dev)
    logits[2] = -float("inf")
    z = block.step(x.to(dev), logits)
    ref = oracle.few_tokens.few_token_moe(f64(x)[2:3], np.full((1, kr), -1), np.zeros((1, kr)), dequantised(w13),
                                          dequantised(w2), (dequantised(shared[0]), dequantised(shared[1])))
    assert oracle.checks.calc_diff(f64(z)[2:3], ref) <= 1e-4
