"""GPU parity of ``swiglu_quantise`` with the float64 oracle.

h is three float32 operations on a float32 exp (2 ulp): within 2**-21 of its
exact value.  So a code is the oracle's code of some value within 2**-21 of h,
and a block exponent the oracle's unless the block's maximum is within 2**-21
of 448 * 2**e.
"""

import numpy as np
import pytest
import torch

import oracle
from block_scaled_fp8_route_gb300 import ops
from tests.gpu_util import bits16, require_gpu, u8

pytestmark = pytest.mark.gpu
DELTA = 2.0 ** -21


@pytest.fixture(scope="module")
def dev():
    return require_gpu()


def _input(T, K, dev, seed=0):
    g = torch.Generator().manual_seed(seed)
    y = torch.randn(T, 2 * K, generator=g) * torch.exp2(torch.randint(-6, 5, (T, 1), generator=g).float())
    return y.to(torch.bfloat16).to(dev)


def _check(y, q, sf, rows=None):
    T, K = y.shape[0], y.shape[1] // 2
    hb = oracle.swiglu.padded_blocks(oracle.swiglu.swiglu(bits16(y)))
    nkb = hb.shape[1]
    e = oracle.quantise.unpack_sf(sf.cpu().numpy(), T, nkb).astype(int) - 127
    amax = np.abs(hb).max(axis=2)
    lo = oracle.quantise._block_exponent(amax * (1 - DELTA))
    hi = oracle.quantise._block_exponent(amax * (1 + DELTA))
    keep = np.ones(T, bool) if rows is None else rows
    assert ((e >= lo) & (e <= hi))[keep].all()
    assert (lo == hi)[keep].mean() > 0.99 or keep.sum() * nkb < 100
    v = oracle.formats.e4m3_decode(u8(q)).reshape(T, nkb, 128)[keep]
    s = np.ldexp(hb, -e[:, :, None])[keep]
    a = oracle.formats.e4m3_decode(oracle.formats.e4m3_encode(s * (1 - DELTA)))
    b = oracle.formats.e4m3_decode(oracle.formats.e4m3_encode(s * (1 + DELTA)))
    assert ((v >= np.minimum(a, b)) & (v <= np.maximum(a, b))).all()
    # bytes of the blocks past Kp in the last word
    words = sf.cpu().numpy().view(np.uint32)[:, :T]
    for j in range(nkb, 4 * words.shape[0]):
        assert (((words[j // 4] >> (8 * (j % 4))) & 0xFF)[keep] == 127).all()


@pytest.mark.parametrize("T", [1, 2, 5, 33, 300])
@pytest.mark.parametrize("K", [8, 64, 120, 128, 136, 512, 520, 1024, 1416, 1536, 2048])
def test_parity(dev, T, K):
    y = _input(T, K, dev, seed=T + K)
    q, sf = ops.swiglu_quantise(y)
    assert q.shape == (T, (K + 127) // 128 * 128)
    _check(y, q, sf)
    assert not u8(q)[:, K:].any()


def test_equals_the_two_call_path_where_h_is_a_bf16_number(dev):
    """g = 128 gives silu(g) = 128 exactly, so h = 128 u is a bf16 value: the same bytes as quantise_act."""
    u = _input(40, 256, dev, seed=2)[:, :256].contiguous()
    y = torch.cat([torch.full_like(u, 128.0), u], dim=1)
    q, sf = ops.swiglu_quantise(y)
    q2, sf2 = ops.quantise_act((u.float() * 128).to(torch.bfloat16))
    assert torch.equal(q, q2) and torch.equal(sf[:, :40], sf2[:, :40])


def test_zero_extreme_and_non_finite_values(dev):
    K = 256
    y = torch.zeros(8, 2 * K)
    y[1, :K] = -200.0                              # silu underflows to a tiny negative number
    y[1, K:] = 3.0
    y[2, :K] = 3.0e38
    y[2, K:] = 1.0
    y[3, :K] = 1e-30
    y[3, K:] = 1e-30                               # h below float32's range
    y[4, :K] = 2.0
    y[4, K:] = torch.arange(K).float() - 128
    yb = y.to(torch.bfloat16).to(dev)
    q, sf = ops.swiglu_quantise(yb)
    _check(yb[[0, 2, 4]], q[[0, 2, 4]], sf[:, [0, 2, 4]])
    assert not (u8(q)[3] & 0x7F).any() and not (u8(q)[1] & 0x7F).any()
    # a NaN stays a NaN code in its own place; its block's scale comes from the other values
    yb[4, 5] = float("nan")
    q2, sf2 = ops.swiglu_quantise(yb)
    assert (u8(q2)[4, 5] & 0x7F) == 0x7F
    q2[4, 5] = q[4, 5]
    assert torch.equal(q2, q) and torch.equal(sf2[:, :8], sf[:, :8])


@pytest.mark.parametrize("layout,amount", [(ops.CONTIGUOUS, 128), (ops.CONTIGUOUS, 1), (ops.MASKED, 16)])
@pytest.mark.parametrize("K", [128, 264])
def test_routed_rows_only(dev, layout, amount, K):
    g = torch.Generator().manual_seed(4)
    ids = torch.stack([torch.randperm(6, generator=g)[:2] for _ in range(37)]).to(torch.int32)
    ids[3] = -1
    r = ops.route(ids.to(dev), 8, layout, amount)
    R = r.m_cap
    y = _input(R, K, dev, seed=5)
    token = r.token_of_row.cpu().numpy()
    used = int(r.seg_start[8])
    keep = (np.arange(R) < used) & (token >= 0)
    y[torch.from_numpy(~keep).to(dev)] = float("nan")
    q = torch.full((R, (K + 127) // 128 * 128), 0x55, dtype=torch.uint8, device=dev)
    sf = torch.full((1, ops.sf_ld(R)), -5, dtype=torch.int32, device=dev)
    ops.swiglu_quantise(y, rows=(r.token_of_row, r.seg_start[8:]), q=q, sf=sf)
    y2 = torch.where(torch.from_numpy(keep).to(dev)[:, None], y, torch.zeros_like(y))
    _check(y2, q, sf, rows=keep)
    assert (u8(q)[~keep] == 0x55).all()
    assert (sf.cpu().numpy()[:, :R][:, ~keep] == -5).all()


@pytest.mark.parametrize("off,extra", [(0, 8), (8, 0), (16, 24)])
def test_row_strides_and_output_bounds(dev, off, extra):
    T, K = 21, 264
    wide = _input(T, K + (off + extra) // 2, dev, seed=6)
    y = wide[:, off:off + 2 * K]
    assert y.stride(0) != 2 * K
    qbuf = torch.full((T + 1, 384), 0xEE, dtype=torch.uint8, device=dev)
    sfbuf = torch.full((1, 24), 99, dtype=torch.int32, device=dev)
    q, sf = ops.swiglu_quantise(y, q=qbuf[:T], sf=sfbuf)
    _check(y.contiguous(), q, sf)
    assert (qbuf[T] == 0xEE).all() and (sfbuf[:, T:] == 99).all()


def test_empty_batch_and_other_stream(dev):
    q, sf = ops.swiglu_quantise(torch.empty(0, 512, dtype=torch.bfloat16, device=dev))
    assert q.shape == (0, 256)
    y = _input(50, 512, dev, seed=7)
    q, sf = ops.swiglu_quantise(y)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    q2, sf2 = ops.swiglu_quantise(y, stream=side)
    side.synchronize()
    assert torch.equal(q, q2) and torch.equal(sf[:, :50], sf2[:, :50])


def test_offsets_past_32_bits(dev):
    """T * ld above 2**31 elements."""
    T, ld, K = 2100, 1 << 20, 128
    y = torch.zeros(T * ld, dtype=torch.bfloat16, device=dev).view(T, ld)[:, :2 * K]
    tail = _input(10, K, dev, seed=8)
    y[-10:] = tail
    q, sf = ops.swiglu_quantise(y)
    q2, sf2 = ops.swiglu_quantise(tail)
    assert torch.equal(q[-10:], q2) and torch.equal(sf[:, T - 10:T], sf2[:, :10])
