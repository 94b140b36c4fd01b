"""MoEBlock end to end against the oracle's whole chain, with a balance bias and groups by their two largest
scores: the same ids, and the E4M3 path's calc_diff threshold on the output (a product that rounds the other
way to bf16 moves a few codes of the next operand, so no bound by element holds over the chain)."""

import numpy as np
import pytest
import torch

import oracle
from block_scaled_fp8_route_gb300 import MoEBlock, ops
from tests.gpu_util import bits16, require_gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,layout,amount", [(1, ops.MASKED, 16), (50, ops.MASKED, 64), (300, ops.CONTIGUOUS, 128)])
@pytest.mark.parametrize("S", [0, 72])
@pytest.mark.parametrize("sigmoid", [True, False])
def test_chain(T, layout, amount, S, sigmoid):
    dev = require_gpu()
    E, kr, K, I, groups, kept = 16, 3, 256, 128, 4, 2
    g = torch.Generator().manual_seed(T + S)
    bf16 = lambda *shape: (torch.randn(*shape, generator=g) * 0.05).to(torch.bfloat16)  # noqa: E731
    w13, w2 = bf16(E, 2 * I, K), bf16(E, K, I)
    shared = (bf16(2 * S, K), bf16(K, S)) if S else None
    x = torch.randn(T, K, generator=g).to(torch.bfloat16)
    # logits and biases in steps, so that no choice hangs on rounding
    logits = torch.stack([torch.randperm(E, generator=g) for _ in range(T)]).float() * 0.37 - 2.5
    bias = torch.randperm(E, generator=g).float() * 0.0131
    block = MoEBlock(E, kr, T, K, I, w13, w2, shared=shared, layout=layout, align_or_max_m=amount, device=dev,
                     score="sigmoid" if sigmoid else "softmax", bias=bias.to(dev), groups=groups, kept_groups=kept,
                     group_score="top2", scale=2.5)
    z = block.step(x.to(dev), logits.to(dev))
    torch.cuda.synchronize()
    assert ops.device_error() == 0
    ref, ids, margin = oracle.block.moe_block(
        bits16(x), logits.numpy(), bits16(w13), bits16(w2), kr, sigmoid=sigmoid, bias=bias.double().numpy(),
        groups=groups, kept=kept, top2=True, scale=2.5, shared=tuple(bits16(w) for w in shared) if S else None)
    clear = margin > 4e-6
    assert clear.mean() > 0.9
    assert np.array_equal(block.topk_ids.cpu().numpy()[clear], ids[clear])
    f = oracle.formats.bf16_bits_to_f64
    assert oracle.checks.calc_diff(f(bits16(z))[clear], f(ref)[clear]) <= oracle.checks.CALC_DIFF_MAX
    for t in np.flatnonzero(clear):
        assert oracle.checks.calc_diff(f(bits16(z))[t], f(ref)[t]) <= oracle.checks.CALC_DIFF_MAX, t
