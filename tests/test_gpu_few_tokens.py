"""GPU parity of ``few_token_moe`` with the float64 oracle, within the derived bound of ``oracle.few_tokens.bound``
plus the rounding of z to bf16 (half a step, 2**-8 of it)."""

import numpy as np
import pytest
import torch

import oracle
from block_scaled_fp8_route_gb300 import ops
from tests.gpu_util import bits16, require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    return require_gpu()


def f64(t):
    return oracle.formats.bf16_bits_to_f64(bits16(t))


class Layer:
    """Random weights of a layer, on the GPU as the operator takes them and in 64 bits."""

    def __init__(self, dev, E, K, I, S=0, fmt="fp8", tiled=True, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.dev, self.E, self.K, self.I, self.S, self.fp8 = dev, E, K, I, S, fmt == "fp8"
        self.flags = ops.B_TILED if tiled else 0

        def make(n, rows, inner):
            w = torch.randn(n, rows, inner, generator=g) * 0.05
            w[:, :, :128] *= 8.0                                     # blocks of different exponents
            w = w.to(torch.bfloat16).to(dev)
            if not self.fp8:
                wide = f64(w)
                return (ops.tile_weights(w) if tiled else w), None, wide
            q, sf128 = ops.quantise_weight(w)
            bq, bsf = oracle.quantise.quantise_weight(bits16(w))
            wide = np.stack([oracle.gemm.dequant_weight(bq[e], bsf[e]) for e in range(n)])
            return (ops.tile_weights(q) if tiled else q), ops.prepare_weight_sf(sf128, inner), wide

        self.w13, self.sf13, self.wide13 = make(E, 2 * I, K)
        self.w2, self.sf2, self.wide2 = make(E, K, I)
        self.shared = self.wide_shared = None
        if S:
            a, b = make(1, 2 * S, K), make(1, K, S)
            self.shared = tuple(None if t is None else t[0] for t in (a[0], a[1], b[0], b[1]))
            self.wide_shared = (a[2][0], b[2][0])

    def call(self, x, ids, p, **kw):
        kw.setdefault("flags", self.flags)
        return ops.few_token_moe(x, ids, p, self.w13, self.sf13, self.w2, self.sf2, shared=self.shared, **kw)

    def check(self, z, x, ids, p, addend=None, rows=None):
        assert ops.device_error() == 0
        args = (f64(x), ids.cpu().numpy(), p.cpu().numpy(), self.wide13, self.wide2, self.wide_shared,
                None if addend is None else f64(addend))
        ref = oracle.few_tokens.few_token_moe(*args)
        tol = oracle.few_tokens.bound(*args, fp8=self.fp8)
        tol = tol + 2.0 ** -8 * (np.abs(ref) + tol)
        got = f64(z)
        rows = slice(None) if rows is None else rows
        bad = ~(np.abs(got - ref) <= tol)[rows]
        worst = np.max((np.abs(got - ref) / np.maximum(tol, 1e-300))[rows], initial=0)
        assert not bad.any(), f"{bad.sum()} of {bad.size} outside, worst {worst:.2f} times the bound"


def inputs(dev, T, K, E, kr, seed=0):
    g = torch.Generator().manual_seed(seed + 100)
    x = torch.randn(T, K, generator=g)
    x[:, torch.rand(K, generator=g) < 0.02] *= 30.0
    ids = torch.stack([torch.randperm(E, generator=g)[:kr] for _ in range(T)]).int()
    p = torch.softmax(torch.randn(T, kr, generator=g), 1)
    return x.to(torch.bfloat16).to(dev), ids.to(dev).contiguous(), p.to(dev)


@pytest.mark.parametrize("fmt", ["fp8", "bf16"])
@pytest.mark.parametrize("T", [1, 2, 7, 8, 9, 16, 17, 24, 25, 31, 32])
def test_tokens(dev, fmt, T):
    layer = Layer(dev, 8, 256, 128, fmt=fmt)
    x, ids, p = inputs(dev, T, 256, 8, 2, T)
    layer.check(layer.call(x, ids, p), x, ids, p)


@pytest.mark.parametrize("fmt", ["fp8", "bf16"])
@pytest.mark.parametrize("E,kr,K,I,S", [(1, 1, 128, 128, 0), (1, 1, 1152, 128, 0), (2, 1, 128, 640, 0),
                                        (33, 5, 640, 384, 128), (256, 8, 896, 128, 384), (16, 16, 384, 256, 0),
                                        (40, 3, 2048, 128, 512), (4, 2, 1920, 640, 0)])
def test_sizes(dev, fmt, E, kr, K, I, S):
    layer = Layer(dev, E, K, I, S, fmt=fmt, seed=E)
    for T in (1, 5, 32):
        x, ids, p = inputs(dev, T, K, E, kr, T)
        layer.check(layer.call(x, ids, p), x, ids, p)


@pytest.mark.parametrize("fmt", ["fp8", "bf16"])
def test_row_major_weights_give_the_same_bits(dev, fmt):
    tiled, rows = (Layer(dev, 6, 384, 256, 128, fmt=fmt, tiled=t) for t in (True, False))
    x, ids, p = inputs(dev, 9, 384, 6, 3)
    assert torch.equal(tiled.call(x, ids, p), rows.call(x, ids, p))


@pytest.mark.parametrize("S", [0, 256])
def test_tokens_without_experts(dev, S):
    layer = Layer(dev, 8, 256, 128, S)
    x, ids, p = inputs(dev, 11, 256, 8, 4)
    ids[2:9] = -1
    ids[9, 1] = -7
    z = layer.call(x, ids, p)
    layer.check(z, x, ids, p)
    ids[:] = -1
    z = layer.call(x, ids, p)
    layer.check(z, x, ids, p)
    if not S:
        assert torch.count_nonzero(z) == 0


def test_every_token_chooses_the_same_experts(dev):
    layer = Layer(dev, 64, 512, 256)
    x, ids, p = inputs(dev, 32, 512, 64, 8)
    ids[:] = ids[0]
    layer.check(layer.call(x, ids, p), x, ids, p)


def test_an_expert_named_twice_counts_with_both_weights(dev):
    layer = Layer(dev, 8, 256, 128)
    x, ids, p = inputs(dev, 13, 256, 8, 4)
    ids[:, 2] = ids[:, 0]
    ids[5] = 3
    layer.check(layer.call(x, ids, p), x, ids, p)


def test_ids_past_the_experts_are_reported_and_skipped(dev):
    layer = Layer(dev, 8, 256, 128)
    x, ids, p = inputs(dev, 6, 256, 8, 2)
    ids[1, 0], ids[4, 1] = 8, 2 ** 31 - 1
    z = layer.call(x, ids, p)
    assert ops.device_error() == ops.DEVERR_EXPERT_ID
    layer.check(z, x, ids, p)


def test_strides_and_addend(dev):
    layer = Layer(dev, 8, 384, 128, 128)
    T, K = 10, 384
    x, ids, p = inputs(dev, T, K, 8, 2)
    wide = torch.full((T, K + 24), float("nan"), dtype=torch.bfloat16, device=dev)
    wide[:, 8:8 + K] = x
    addend = torch.randn(T, K + 3, device=dev).to(torch.bfloat16)[:, 1:1 + K]
    out = torch.full((T + 2, K + 5), 7.0, dtype=torch.bfloat16, device=dev)
    z = out[1:1 + T, 3:3 + K]
    assert layer.call(wide[:, 8:8 + K], ids, p, addend=addend, z=z).data_ptr() == z.data_ptr()
    layer.check(z, x, ids, p, addend)
    z_plain = z.clone()
    z.fill_(7.0)
    assert torch.all(out == 7.0)                                     # nothing around z was written
    same = addend.contiguous()
    layer.call(x, ids, p, addend=same, z=same)                       # onto the addend itself, other strides
    assert torch.equal(same, z_plain)


def test_values_far_apart_in_a_block(dev):
    """Rows whose values span 2**40, tiny ones, zeros: the split's tail and its clamped exponents."""
    layer = Layer(dev, 4, 256, 128)
    x, ids, p = inputs(dev, 8, 256, 4, 2)
    g = torch.Generator().manual_seed(5)
    x[0] *= torch.exp2(torch.randint(-40, 1, (256,), generator=g).float()).to(dev)
    x[1] = 0
    x[2, :128] = 0
    x[3] *= 2.0 ** -100
    x[4] = torch.finfo(torch.bfloat16).tiny
    x[5] *= 2.0 ** 20
    layer.check(layer.call(x, ids, p), x, ids, p)


@pytest.mark.parametrize("fmt", ["fp8", "bf16"])
def test_not_finite_inputs_stay_in_their_row(dev, fmt):
    layer = Layer(dev, 8, 256, 128, 128, fmt=fmt)
    x, ids, p = inputs(dev, 12, 256, 8, 2)
    x[3, 17], x[5, 200], x[7, 0] = float("inf"), float("nan"), -float("inf")
    p[9, 1] = float("nan")
    z = layer.call(x, ids, p)
    assert ops.device_error() == 0
    for t in (3, 5, 7, 9):
        assert not torch.isfinite(z[t]).any()
    x[3], x[5], x[7], p[9] = 0, 0, 0, 0
    rest = [t for t in range(12) if t not in (3, 5, 7, 9)]
    layer.check(z, x, ids, p, rows=rest)


def test_same_bits_every_run_and_in_a_graph(dev):
    layer = Layer(dev, 32, 1024, 384, 256)
    T = 19
    x, ids, p = inputs(dev, T, 1024, 32, 4)
    ws = ops.few_token_moe_workspace(T, 4, 384, 256, device=dev)
    ws.fill_(255)                                                    # any contents
    z = layer.call(x, ids, p, workspace=ws).clone()
    layer.check(z, x, ids, p)
    out = torch.empty_like(z)
    for _ in range(20):
        assert torch.equal(layer.call(x, ids, p, workspace=ws, z=out), z)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.call(x, ids, p, workspace=ws, z=out)
    x2, ids2, p2 = inputs(dev, T, 1024, 32, 4, seed=9)
    for src, a, b, c in ((z, x.clone(), ids.clone(), p.clone()), (layer.call(x2, ids2, p2).clone(), x2, ids2, p2)):
        x.copy_(a), ids.copy_(b), p.copy_(c)
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, src)


def test_back_to_back_calls_and_other_streams(dev):
    """Calls queued without a pause on one workspace, and calls on two streams with one each."""
    layer = Layer(dev, 16, 512, 256)
    cases = [inputs(dev, T, 512, 16, 3, seed=T) for T in (1, 32, 5, 16, 9, 27)]
    want = [layer.call(*c).clone() for c in cases]
    torch.cuda.synchronize()
    ws = ops.few_token_moe_workspace(32, 3, 256, device=dev)
    got = [layer.call(*c, workspace=ws) for c in cases * 5]
    torch.cuda.synchronize()
    for i, z in enumerate(got):
        assert torch.equal(z, want[i % len(cases)])
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [layer.call(*c, stream=streams[i % 2]) for i, c in enumerate(cases * 4)]
    torch.cuda.synchronize()
    for i, z in enumerate(got):
        assert torch.equal(z, want[i % len(cases)])


def test_a_wait_that_runs_out(dev):
    layer = Layer(dev, 8, 256, 128)
    x, ids, p = inputs(dev, 5, 256, 8, 2)
    want = layer.call(x, ids, p)
    z = torch.full_like(want, 3.0)
    layer.call(x, ids, p, z=z, flags=ops.B_TILED | 0x100)
    assert ops.device_error() == ops.DEVERR_TIMEOUT
    assert torch.all(torch.isnan(z) | (z == 3.0))
    assert torch.equal(layer.call(x, ids, p), want)
    assert ops.device_error() == 0


def test_no_tokens(dev):
    layer = Layer(dev, 4, 256, 128, 128)
    x, ids, p = inputs(dev, 3, 256, 4, 2)
    z = layer.call(x[:0], ids[:0], p[:0])
    assert z.shape == (0, 256) and ops.device_error() == 0


def test_graph_and_eager_calls_that_allocate_their_own_workspace(dev):
    """Two captured calls and eager ones in between, none with a workspace of the caller's."""
    layer = Layer(dev, 16, 512, 256, 128)
    cases = [inputs(dev, T, 512, 16, 3, seed=T) for T in (4, 29)]
    want = [layer.call(*c).clone() for c in cases]
    graphs = []
    for c in cases:
        z = torch.empty_like(c[0])
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            layer.call(*c, z=z)
            layer.call(*c, z=z)
        graphs.append((g, z))
    for _ in range(5):
        for (g, z), c, w in zip(graphs, cases, want):
            z.zero_()
            g.replay()
            other = [torch.empty(1 << 16, dtype=torch.uint8, device=dev).fill_(255) for _ in range(4)]
            assert torch.equal(layer.call(*c), w)
            torch.cuda.synchronize()
            assert torch.equal(z, w) and len(other) == 4


def test_more_experts_than_a_table_of_one_warp(dev):
    """1024 experts, as many as there may be, most of them chosen by nobody or by one token."""
    layer = Layer(dev, 1024, 128, 128, seed=1)
    x, ids, p = inputs(dev, 32, 128, 1024, 32, 7)
    ids[0, 0], ids[31, 31] = 0, 1023
    layer.check(layer.call(x, ids, p), x, ids, p)


@pytest.mark.parametrize("K,I,S", [(2176, 128, 0), (2048, 1408, 2816)])
def test_second_products_in_pairs_of_tiles(dev, K, I, S):
    """Wide enough for two tiles of W2 a CTA, also where their number is odd, with a heavy shared expert."""
    layer = Layer(dev, 6, K, I, S)
    for T in (2, 16):
        x, ids, p = inputs(dev, T, K, 6, 2, T)
        layer.check(layer.call(x, ids, p), x, ids, p)


@pytest.mark.parametrize("fmt", ["fp8", "bf16"])
@pytest.mark.parametrize("T", [9, 17, 25, 32])
def test_a_heavy_expert_among_light_ones(dev, fmt, T):
    """Experts of 9 tokens and more cost the first kernel more than one unit: one that all choose, first, in the middle or
    last, some of about half the tokens, and a shared one."""
    for heavy, S in ((0, 0), (9, 256), (19, 128)):
        layer = Layer(dev, 20, 640, 256, S, fmt=fmt, seed=heavy)
        x, ids, p = inputs(dev, T, 640, 20, 3, seed=T + heavy)
        ids[:, 1] = heavy
        ids[:T // 2 + 1, 2] = (heavy + 7) % 20
        layer.check(layer.call(x, ids, p), x, ids, p)


def test_many_heavy_experts(dev):
    """1024 assignments in groups of nine tokens an expert, as many costs beyond one as there can be, on 1024 experts."""
    layer = Layer(dev, 1024, 128, 128, seed=3)
    x, ids, p = inputs(dev, 32, 128, 1024, 32, 3)
    free = [0] * 32
    for e in range(113):
        order = sorted(range(32), key=lambda t: (free[t], t))[:9]
        for t in order:
            if free[t] < 32:
                ids[t, free[t]] = 9 * e + 3
                free[t] += 1
    layer.check(layer.call(x, ids, p), x, ids, p)


@pytest.mark.parametrize("fmt", ["fp8", "bf16"])
@pytest.mark.parametrize("T", [1, 2, 5, 10, 17, 32])
@pytest.mark.parametrize("E,I,S", [(1, 128, 0), (1, 256, 0), (1, 512, 0), (3, 128, 128), (4, 384, 0)])
def test_few_blocks_and_many_tokens(dev, fmt, T, E, I, S):
    """One to a few K-blocks a CTA of the second kernel, so that 8, 4 or 2 warps form one; some tokens choose nothing."""
    layer = Layer(dev, E, 384, I, S, fmt=fmt, seed=I)
    x, ids, p = inputs(dev, T, 384, E, min(2, E), seed=T)
    if T > 4:
        ids[1] = -1
        ids[T - 1] = -1
    layer.check(layer.call(x, ids, p), x, ids, p)
