"""GPU parity of ``dense_gemm`` with the float64 oracle.

Bound per element: the bf16 rounding of the result, 2**-8 |ref| (half a step is
2**-9; the other half covers a sum that moved across a power of two), plus the
tensor core's float32 accumulation, K / 32 instructions of at most four
roundings each of the running sum of magnitudes S = sum |a b| (+ |c|):
K / 8 * 2**-24 * S.
"""

import numpy as np
import pytest
import torch

import oracle
from block_scaled_fp8_route_gb300 import ops
from tests.gpu_util import bits16, require_gpu, u8

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    return require_gpu()


class Problem:
    def __init__(self, M, N, K, dev, seed=0, addend=False):
        g = torch.Generator().manual_seed(seed)
        self.M, self.N, self.K = M, N, K
        x = torch.randn(M, K, generator=g) * torch.exp2(torch.randint(-4, 5, (M, 1), generator=g).float())
        self.x = x.to(torch.bfloat16).to(dev)
        w = torch.randn(N, K, generator=g) * 0.02
        w[:, :128] *= 64.0                                       # blocks of different exponents
        self.w = w.to(torch.bfloat16).to(dev)
        self.a, self.sfa = ops.quantise_act(self.x)
        self.b, self.sfb = ops.prepare_dense_weight(self.w)
        self.c = torch.randn(M, N, generator=g).to(torch.bfloat16).to(dev) if addend else None

    def reference(self):
        """(ref float64, sum of magnitudes) from the oracle's own quantisation of x and w."""
        aq, asf = oracle.quantise.quantise_act(bits16(self.x))
        pad = torch.nn.functional.pad(self.w, (0, 0, 0, -self.N % 128))
        bq, bsf = oracle.quantise.quantise_weight(bits16(pad)[None])
        a = oracle.gemm.dequant_rows(aq, asf)
        b = oracle.gemm.dequant_weight(bq[0], bsf[0])[:self.N]
        ref, mag = a @ b.T, np.abs(a) @ np.abs(b).T
        if self.c is not None:
            c = oracle.formats.bf16_bits_to_f64(bits16(self.c))
            ref, mag = ref + c, mag + np.abs(c)
        return ref, mag

    def check(self, d, what=""):
        ref, mag = self.reference()
        v = oracle.formats.bf16_bits_to_f64(bits16(d))
        bound = 2.0 ** -8 * np.abs(ref) + self.K / 8 * 2.0 ** -24 * mag
        bad = ~(np.abs(v - ref) <= bound)
        assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} outside, first at {np.argwhere(bad)[:4].tolist()}"

    def run(self, **kw):
        return ops.dense_gemm(self.a, self.sfa, self.b, self.sfb, self.N, addend=self.c, **kw)


@pytest.mark.parametrize("M", [1, 2, 15, 16, 17, 31, 33, 64, 65, 128, 129, 200, 255, 256, 257, 300, 513, 1000])
@pytest.mark.parametrize("N,K", [(128, 128), (256, 640), (384, 1024)])
def test_token_counts(dev, M, N, K):
    p = Problem(M, N, K, dev, seed=M + K, addend=M % 2 == 1)
    p.check(p.run(), f"M={M}")


@pytest.mark.parametrize("N", [1, 7, 8, 100, 127, 129, 130, 200, 252, 320, 576, 1000, 2112])
@pytest.mark.parametrize("M", [1, 37, 290])
def test_output_widths(dev, N, M):
    p = Problem(M, N, 512, dev, seed=N, addend=True)
    p.check(p.run(), f"N={N}")


@pytest.mark.parametrize("K", [128, 256, 384, 512, 640, 896, 1152, 2048, 2176, 4096, 7168])
@pytest.mark.parametrize("M", [3, 150])
def test_inner_lengths(dev, K, M):
    p = Problem(M, 256, K, dev, seed=K)
    p.check(p.run(), f"K={K}")


# (sizes that reach every tile of the CTA pairs: 224, 192, 160 and 128 tokens, one tile per pair and several,
# odd counts of 128-row weight tiles and of K-blocks)
@pytest.mark.parametrize("M,N,K", [(2048, 1536, 512), (1500, 2304, 1024), (4100, 640, 256), (513, 4096, 384),
                                   (777, 4096, 2048), (1500, 4096, 896), (640, 4096, 1152), (4700, 1100, 2048),
                                   (1024, 7168, 640), (5000, 4096, 128)])
def test_larger_products(dev, M, N, K):
    p = Problem(M, N, K, dev, seed=M, addend=True)
    p.check(p.run())


# (tiles of 96 and 128 tokens, which two warps multiply: one tile per pair and several, inner lengths of 2 to 57
# blocks, a last tile of few tokens, a last weight tile of 4 rows)
@pytest.mark.parametrize("M,N,K", [(300, 4096, 4096), (500, 4096, 7296), (520, 2112, 2176), (910, 4100, 1152),
                                   (1230, 4096, 640), (970, 7168, 256), (1235, 4096, 384), (2600, 7168, 256)])
@pytest.mark.parametrize("addend", [False, True])
def test_products_in_narrow_pair_tiles(dev, M, N, K, addend):
    p = Problem(M, N, K, dev, seed=M + N, addend=addend)
    first = p.run()
    p.check(first)
    assert torch.equal(p.run(), first)


def test_row_major_weights_give_the_same_bits(dev):
    for M in (5, 260, 2050):
        p = Problem(M, 300, 640, dev, seed=1)
        wq, sf128 = ops.quantise_weight(torch.nn.functional.pad(p.w, (0, 0, 0, -300 % 128)).unsqueeze(0))
        d = ops.dense_gemm(p.a, p.sfa, wq[0], p.sfb, 300, flags=0)
        assert torch.equal(d, p.run())


@pytest.mark.parametrize("off,extra,coff,cextra", [(0, 4, 0, 0), (1, 2, 0, 3), (3, 8, 1, 1), (4, 12, 4, 4),
                                                   (8, 8, 8, 16), (2, 6, 0, 0)])
@pytest.mark.parametrize("M,N", [(19, 200), (300, 256), (2100, 328)])
def test_strides_alignment_and_bounds(dev, off, extra, coff, cextra, M, N):
    """d and addend as windows of wider tensors: the window is right, nothing around it is written."""
    p = Problem(M, N, 256, dev, seed=off + N, addend=True)
    want = p.run()
    wide_c = torch.full((M, N + coff + cextra), 5.0, dtype=torch.bfloat16, device=dev)
    wide_c[:, coff:coff + N] = p.c
    wide_d = torch.full((M + 2, N + off + extra), -3.0, dtype=torch.bfloat16, device=dev)
    d = wide_d[1:M + 1, off:off + N]
    ops.dense_gemm(p.a, p.sfa, p.b, p.sfb, N, addend=wide_c[:, coff:coff + N], d=d)
    assert torch.equal(d, want)
    wide_d[1:M + 1, off:off + N] = -3.0
    assert (wide_d == -3.0).all()


@pytest.mark.parametrize("M,N,K", [(300, 4090, 2048), (1300, 2113, 512), (2100, 1541, 256), (900, 4095, 640),
                                   (40, 1001, 256), (129, 27, 128)])
@pytest.mark.parametrize("addend", [False, True])
def test_columns_past_n_are_not_written(dev, M, N, K, addend):
    """16-byte aligned rows of a width that is not a multiple of 8: what lies behind them stays."""
    p = Problem(M, N, K, dev, seed=N, addend=addend)
    wide = torch.full((M + 1, N + 8 + -N % 8), 7.0, dtype=torch.bfloat16, device=dev)
    if addend:                                                   # the addend's rows are aligned too
        c = torch.full((M, N + -N % 8), float("nan"), dtype=torch.bfloat16, device=dev)
        c[:, :N] = p.c
        p.c = c[:, :N]
    d = p.run(d=wide[:M, :N])
    p.check(d)
    assert (wide[:M, N:] == 7.0).all() and (wide[M] == 7.0).all()


def test_addend_may_be_the_output(dev):
    for M in (9, 1100):
        p = Problem(M, 512, 384, dev, seed=3, addend=True)
        want = p.run()
        d = p.c.clone()
        ops.dense_gemm(p.a, p.sfa, p.b, p.sfb, 512, addend=d, d=d)
        assert torch.equal(d, want)


def test_repeat_runs_are_bit_identical_and_streams(dev):
    for M in (1, 70, 777, 2304):
        p = Problem(M, 1024, 2048, dev, seed=4)
        want = p.run()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        for i in range(20):
            d = p.run(stream=side if i % 2 else None)
            torch.cuda.synchronize()
            assert torch.equal(d, want)
    assert ops.device_error() == 0


def test_equals_the_grouped_product_with_one_expert_to_the_last_sum(dev):
    """The grouped product of one expert on the same operands: within the same bound of each other."""
    p = Problem(300, 512, 1024, dev, seed=5)
    seg = torch.tensor([0, 300], dtype=torch.int32, device=dev)
    cnt = torch.tensor([300], dtype=torch.int32, device=dev)
    g = ops.grouped_gemm_contig(p.a, p.sfa, p.b.unsqueeze(0), p.sfb.unsqueeze(0), seg, cnt, flags=ops.B_TILED)
    p.check(g, "grouped")
    p.check(p.run(), "dense")


def test_infinite_and_nan_operands_stay_in_their_rows(dev):
    p = Problem(40, 256, 256, dev, seed=6)
    want = p.run()
    p.a[7, 3] = 0x7F                                             # an E4M3 NaN
    d = p.run()
    assert torch.isnan(d[7]).all()
    d[7] = want[7]
    assert torch.equal(d, want)


def test_wide_scale_range(dev):
    """Block exponents from 2**-60 to 2**60 in one row."""
    g = torch.Generator().manual_seed(11)
    x = torch.randn(20, 512, generator=g) * torch.exp2(torch.tensor([-60.0, -3.0, 0.0, 60.0])).repeat_interleave(128)
    p = Problem(20, 256, 512, dev, seed=11)
    p.x = x.to(torch.bfloat16).to(dev)
    p.a, p.sfa = ops.quantise_act(p.x)
    p.check(p.run())


def test_empty_batch(dev):
    p = Problem(4, 128, 128, dev)
    d = ops.dense_gemm(p.a[:0], p.sfa, p.b, p.sfb, 128)
    assert d.shape == (0, 128)


def test_offsets_past_32_bits(dev):
    """M * ldd above 2**31 elements."""
    p = Problem(2100, 128, 128, dev, seed=12)
    want = p.run()
    big = torch.empty(2100 << 20, dtype=torch.bfloat16, device=dev).view(2100, 1 << 20)
    d = ops.dense_gemm(p.a, p.sfa, p.b, p.sfb, 128, d=big[:, :128])
    assert torch.equal(d, want)


@pytest.mark.parametrize("M,N,K", [(40, 256, 2048), (300, 512, 256), (2048, 1536, 512)])
def test_withheld_loads_time_out_and_context_survives(dev, M, N, K):
    """The loads never come: every wait of either kernel runs out, the error word says so, nothing is stored,
    and the next product is right."""
    p = Problem(M, N, K, dev, seed=21)
    want = p.run()
    torch.cuda.synchronize()
    assert ops.device_error() == 0
    d = torch.full((M, N), 7.0, dtype=torch.bfloat16, device=dev)
    p.run(d=d, flags=ops.B_TILED | 0x100)
    torch.cuda.synchronize()
    assert ops.device_error() & ops.DEVERR_TIMEOUT
    assert (d == 7.0).all()
    assert torch.equal(p.run(), want)
    assert ops.device_error() == 0


@pytest.mark.parametrize("M,N,K", [(300, 4096, 2048), (1230, 4096, 640)])
def test_withheld_loads_stop_both_issuers_of_a_pair(dev, M, N, K):
    """Tiles of 96 tokens, one and several per pair: neither issuing warp is left at its barrier."""
    test_withheld_loads_time_out_and_context_survives(dev, M, N, K)
