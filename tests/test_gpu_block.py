"""MoEBlock: every stage against the oracle on the stage before it as the GPU left it, so that each is
checked under its own bound, and the block's graph against its eager step."""

import numpy as np
import pytest
import torch

import oracle
from block_scaled_fp8_route_gb300 import MoEBlock, ops
from tests.gpu_util import bits16, check_combine_of_own_y, check_expert_block, require_gpu, u8

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    return require_gpu()


def _weights(E, K, I, S, seed):
    g = torch.Generator().manual_seed(seed)
    w13 = (torch.randn(E, 2 * I, K, generator=g) * 0.05).to(torch.bfloat16)
    w2 = (torch.randn(E, K, I, generator=g) * 0.05).to(torch.bfloat16)
    shared = None
    if S:
        shared = ((torch.randn(2 * S, K, generator=g) * 0.05).to(torch.bfloat16),
                  (torch.randn(K, S, generator=g) * 0.05).to(torch.bfloat16))
    return w13, w2, shared


def _inputs(T, K, E, seed, dtype=torch.float32):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(T, K, generator=g).to(torch.bfloat16), torch.randn(T, E, generator=g).to(dtype)


def _grouped_rows(path, q, sf, w_bf16, seg, counts):
    """Oracle of a grouped GEMM on the GPU's packed operand (its routed rows)."""
    nkb = q.shape[1] // 128
    sfb = oracle.quantise.unpack_sf(sf.cpu().numpy(), q.shape[0], nkb)
    bq, bsf = oracle.quantise.quantise_weight(bits16(w_bf16))
    return oracle.gemm.grouped_gemm(u8(q), sfb, bq, bsf, seg, counts)[0]


def _dense(q, sf, w, rows):
    pad = torch.nn.functional.pad(w, (0, -w.shape[1] % 128, 0, -w.shape[0] % 128))
    bq, bsf = oracle.quantise.quantise_weight(bits16(pad)[None])
    a = oracle.gemm.dequant_rows(u8(q), oracle.quantise.unpack_sf(sf.cpu().numpy(), rows, q.shape[1] // 128))
    b = oracle.gemm.dequant_weight(bq[0], bsf[0])[:w.shape[0]]
    return a @ b.T, np.abs(a) @ np.abs(b).T


@pytest.mark.parametrize("T,layout,amount", [(1, ops.MASKED, 16), (37, ops.MASKED, 64), (64, ops.CONTIGUOUS, 1),
                                             (300, ops.CONTIGUOUS, 128), (3000, ops.CONTIGUOUS, 128)])
@pytest.mark.parametrize("S", [0, 200])
def test_stages(dev, T, layout, amount, S):
    E, kr, K, I = 8, 2, 256, 128
    w13, w2, shared = _weights(E, K, I, S, T)
    x, logits = _inputs(T, K, E, T + 1)
    if T > 10:
        logits[3] = -float("inf")                                 # a token that no routed expert takes
    block = MoEBlock(E, kr, T, K, I, w13, w2, shared=shared, layout=layout, align_or_max_m=amount, device=dev,
                     score="sigmoid", groups=4, kept_groups=2, scale=2.0)
    if S:
        routed_only = MoEBlock(E, kr, T, K, I, w13, w2, layout=layout, align_or_max_m=amount, device=dev,
                               score="sigmoid", groups=4, kept_groups=2, scale=2.0).step(x.to(dev), logits.to(dev))
        routed_only = bits16(routed_only)
    xd, ld = x.to(dev), logits.to(dev)
    z = block.step(xd, ld)
    torch.cuda.synchronize()
    assert ops.device_error() == 0
    p, b = block.path, block.path.bufs

    ids, weights, _ = oracle.gate.gate(logits.numpy(), kr, sigmoid=True, groups=4, kept=2, scale=2.0)
    assert np.array_equal(block.topk_ids.cpu().numpy(), ids)
    np.testing.assert_allclose(block.topk_weights.cpu().numpy(), weights, rtol=2e-6)
    r = oracle.route.route(ids, E, layout, **({"align": amount} if layout == ops.CONTIGUOUS else {"max_m": amount}))
    counts, seg = np.asarray(r["counts"]), np.asarray(r["seg_start"])
    assert np.array_equal(b.counts.cpu().numpy(), counts)

    y_ref = _grouped_rows(p, b.a_packed, b.sfa_packed, w13, seg, counts)
    y, y2 = bits16(p.y), bits16(p.y2)
    y2_ref = _grouped_rows(p, p.q2, p.sf2, w2, seg, counts)
    hb = oracle.swiglu.padded_blocks(oracle.swiglu.swiglu(y))
    e2 = oracle.quantise.unpack_sf(p.sf2.cpu().numpy(), p.q2.shape[0], 1).astype(int) - 127
    for e in range(E):
        rows = slice(int(seg[e]), int(seg[e]) + int(counts[e]))
        if counts[e] == 0:
            continue
        check_expert_block(y[rows], y_ref[rows], f"gate-up, expert {e}")
        s = np.ldexp(hb[rows], -e2[rows][:, :, None])
        assert (np.abs(s).max(axis=2) <= 448 * (1 + 2.0 ** -21)).all()
        lo = oracle.formats.e4m3_decode(oracle.formats.e4m3_encode(s * (1 - 2.0 ** -21)))
        hi = oracle.formats.e4m3_decode(oracle.formats.e4m3_encode(s * (1 + 2.0 ** -21)))
        v = oracle.formats.e4m3_decode(u8(p.q2)[rows]).reshape(s.shape)
        assert ((v >= np.minimum(lo, hi)) & (v <= np.maximum(lo, hi))).all()
        check_expert_block(y2[rows], y2_ref[rows], f"down, expert {e}")
    zb = bits16(z) if not S else routed_only
    check_combine_of_own_y(zb, y2, b.output_index.cpu().numpy(), block.topk_weights.cpu().numpy(), "combine")
    if T > 10:
        assert not zb[3].any()
    if S:
        ref, mag = _dense(p.q, p.sf, shared[0], T)
        got = oracle.formats.bf16_bits_to_f64(bits16(block.shared_y))
        assert (np.abs(got - ref) <= 2.0 ** -8 * np.abs(ref) + K / 8 * 2.0 ** -24 * mag).all()
        ref, mag = _dense(block.shared_q, block.shared_sf, shared[1], T)
        c = oracle.formats.bf16_bits_to_f64(routed_only)
        got = oracle.formats.bf16_bits_to_f64(bits16(z))
        bound = 2.0 ** -8 * np.abs(ref + c) + 256 / 8 * 2.0 ** -24 * (mag + np.abs(c))
        assert (np.abs(got - (ref + c)) <= bound).all()


@pytest.mark.parametrize("T,layout,amount", [(5, ops.MASKED, 16), (700, ops.CONTIGUOUS, 128)])
def test_graph_replay_follows_its_inputs(dev, T, layout, amount):
    E, kr, K, I = 8, 2, 256, 128
    w13, w2, shared = _weights(E, K, I, 136, 3)
    x, logits = (t.to(dev) for t in _inputs(T, K, E, 4, torch.bfloat16))
    block = MoEBlock(E, kr, T, K, I, w13, w2, shared=shared, layout=layout, align_or_max_m=amount, device=dev)
    block.capture(x, logits)
    for seed in (5, 6, 7):
        x2, l2 = _inputs(T, K, E, seed, torch.bfloat16)
        x.copy_(x2)
        logits.copy_(l2)
        got = block.replay().clone()
        want = block.step(x, logits, z=torch.empty_like(block.z))
        assert torch.equal(got, want)


def test_refuses_weights_of_other_shapes(dev):
    w13, w2, shared = _weights(4, 256, 128, 64, 1)
    with pytest.raises(ValueError, match="w13"):
        MoEBlock(4, 2, 8, 256, 128, w13[:, :128], w2, device=dev)
    with pytest.raises(ValueError, match="shared"):
        MoEBlock(4, 2, 8, 256, 128, w13, w2, shared=(shared[0], shared[1][:, :32]), device=dev)
