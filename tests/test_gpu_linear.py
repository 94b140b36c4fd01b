"""GPU parity of ``linear`` with the float64 oracle, within ``oracle.linear.bound``."""

import numpy as np
import pytest
import torch

import oracle
from block_scaled_fp8_route_gb300 import ops
from tests.gpu_util import require_gpu

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
EPS = {BF16: 2.0 ** -8, F16: 2.0 ** -11, F32: 2.0 ** -24}
TINY = {BF16: 2.0 ** -134, F16: 2.0 ** -25, F32: 2.0 ** -150}


@pytest.fixture(scope="module")
def dev():
    return require_gpu()


def wide(t):
    return None if t is None else t.double().cpu().numpy()


class Problem:
    def __init__(self, dev, T, N, K, dtype=BF16, out=None, bias=None, act=None, residual=False, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.act, self.out = act, out or dtype
        self.x = (torch.randn(T, K, generator=g) * torch.exp2(torch.randint(-3, 4, (T, 1), generator=g).float())).to(dtype)
        self.w = (torch.randn(N, K, generator=g) / K ** 0.5).to(dtype)
        self.bias = None if bias is None else torch.randn(N, generator=g).to(bias)
        self.residual = torch.randn(T, N, generator=g).to(self.out) if residual else None
        self.x, self.w, self.bias, self.residual = (None if t is None else t.to(dev) for t in
                                                    (self.x, self.w, self.bias, self.residual))

    def run(self, **kw):
        kw.setdefault("out_dtype", self.out)
        kw.setdefault("residual", self.residual)
        return ops.linear(self.x, self.w, bias=self.bias, activation=self.act, **kw)

    def check(self, y):
        assert ops.device_error() == 0
        args = (wide(self.x), wide(self.w), wide(self.bias), self.act, wide(self.residual))
        ref = oracle.linear.linear(*args)
        tol = oracle.linear.bound(*args, eps=EPS[self.out], tiny=TINY[self.out])
        got = wide(y)
        bad = ~(np.abs(got - ref) <= tol)
        assert not bad.any(), (f"{bad.sum()} of {bad.size} outside, first {np.argwhere(bad)[:3].tolist()}, worst "
                               f"{np.nanmax(np.abs(got - ref) / tol):.2f} times the bound")


@pytest.mark.parametrize("dtype,out", [(BF16, BF16), (BF16, F32), (BF16, F16), (F16, F16), (F16, F32), (F16, BF16)])
@pytest.mark.parametrize("T", [1, 3, 16, 17, 64, 65, 128, 129, 300, 1000])
def test_tokens_and_types(dev, dtype, out, T):
    p = Problem(dev, T, 200, 328, dtype, out, bias=F32, act="silu", residual=True, seed=T)
    p.check(p.run())


# widths and lengths around every tile: 128 rows, 64 values, one block, K that is no multiple of 8
@pytest.mark.parametrize("T,N,K", [(1, 1, 1), (2, 8, 8), (5, 127, 63), (33, 129, 65), (70, 255, 128), (200, 257, 130),
                                   (129, 384, 1000), (4, 4096, 2048), (1, 256, 7168), (512, 256, 4096), (640, 1031, 520),
                                   (2500, 514, 72), (1, 9000, 40), (3000, 1, 500), (513, 2048, 100)])
@pytest.mark.parametrize("out", [BF16, F32])
def test_sizes(dev, T, N, K, out):
    Kp = (K + 7) // 8 * 8
    p = Problem(dev, T, N, Kp, BF16, out, bias=BF16, residual=True, seed=N)
    p.x, p.w = p.x[:, :K], p.w[:, :K]                                # rows strided past K
    p.check(p.run())


@pytest.mark.parametrize("act", ["relu", "silu", "gelu", "gelu_tanh", "sigmoid", None])
@pytest.mark.parametrize("T", [7, 1500])
@pytest.mark.parametrize("out", [F32, F16])
def test_activations(dev, act, T, out):
    p = Problem(dev, T, 520, 264, F16, out, bias=F16, act=act)
    p.check(p.run())


@pytest.mark.parametrize("T", [6, 700])
@pytest.mark.parametrize("act", ["relu", "silu", "gelu", "gelu_tanh", "sigmoid"])
def test_tails_of_the_activations(dev, act, T):
    """One-term sums: v is the bias alone, from -60 to 60, and the result has to be right relative to its size."""
    N = 512
    x, w = torch.zeros(T, 64, dtype=BF16, device=dev), torch.zeros(N, 64, dtype=BF16, device=dev)
    bias = torch.linspace(-60, 60, N, device=dev)
    y = wide(ops.linear(x, w, bias=bias, activation=act, out_dtype=F32))
    ref = oracle.linear.activate(wide(bias), act)
    # exp(-v) and erfc carry an argument rounded by 2**-24 of |v| <= 60 (squared in the gelus: v^2 or v^3 of it)
    tol = 60 ** 3 * 2.0 ** -24 * np.abs(ref) + 2.0 ** -118
    assert np.all(np.abs(y - ref) <= tol)


@pytest.mark.parametrize("T", [9, 1200])
@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("N", [256, 250, 251])
def test_strides_offsets_and_the_output_onto_its_residual(dev, T, out, N):
    p = Problem(dev, T, N, 200, BF16, out, bias=F32, act="gelu", residual=True)
    xs = torch.full((T, 232), float("nan"), dtype=BF16, device=dev)
    xs[:, 16:216] = p.x
    ws = torch.full((N + 4, 208), float("nan"), dtype=BF16, device=dev)
    ws[2:-2, :200] = p.w
    want = p.run()
    p.check(want)
    p.x, p.w = xs[:, 16:216], ws[2:-2, :200]
    for left, pitch in ((0, N + 8), (1, N + 3), (3, N + 5), (4, N + 4)):
        buf = torch.full((T + 2, pitch), 7.0, dtype=out, device=dev)
        y = buf[1:1 + T, left:left + N]
        y.copy_(p.residual)
        p.run(out=y, residual=y)
        assert torch.equal(y, want)
        y.fill_(7.0)
        assert torch.all(buf == 7.0)                                 # nothing around y was written


def test_the_stride_of_a_single_row_is_not_looked_at(dev):
    p = Problem(dev, 1, 300, 128, bias=F32)
    want = p.run()
    base = torch.empty(1, 128 * 3 + 1, dtype=BF16, device=dev)       # row stride 385
    base[:, :128] = p.x
    p.x = base[:, :128]
    assert torch.equal(p.run(), want)


@pytest.mark.parametrize("T", [5, 900])
def test_not_finite_values(dev, T):
    p = Problem(dev, T, 192, 128, BF16, F32, residual=True)
    p.x[2, 5], p.x[3, 7] = float("nan"), float("inf")
    p.w[10] = 0.0
    p.w[11, 7] = float("-inf")
    y = p.run()
    ref = p.x.float() @ p.w.float().t() + p.residual
    assert torch.equal(torch.isnan(y), torch.isnan(ref))
    assert torch.equal(torch.isinf(y), torch.isinf(ref))
    assert torch.isnan(y[2]).all() and not torch.isfinite(y[:, 11]).any()
    for act in ("relu", "silu", "gelu", "sigmoid"):
        a = ops.linear(p.x, p.w, activation=act, out_dtype=F32)
        assert torch.isnan(a[2]).all()
    ok = [t for t in range(T) if t not in (2, 3)]
    cols = [n for n in range(192) if n != 11]
    clean = Problem(dev, T, 192, 128, BF16, F32, residual=True)
    clean.w[10] = 0.0
    assert torch.equal(clean.run()[ok][:, cols], y[ok][:, cols])


def test_half_precision_overflows_to_infinity(dev):
    x = torch.full((3, 64), 200.0, dtype=F16, device=dev)
    w = torch.full((40, 64), 100.0, dtype=F16, device=dev)
    assert torch.isinf(ops.linear(x, w)).all()
    assert torch.all(ops.linear(x, w, out_dtype=F32) == 200.0 * 100.0 * 64)


@pytest.mark.parametrize("T,N,K", [(1, 512, 4096), (100, 384, 2048), (3000, 777, 1032)])
def test_same_bits_every_run_and_in_a_graph(dev, T, N, K):
    p = Problem(dev, T, N, K, BF16, BF16, bias=F32, act="silu", residual=True)
    want = p.run()
    p.check(want)
    out = torch.empty_like(want)
    for _ in range(10):
        assert torch.equal(p.run(out=out), want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        p.run(out=out)
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [p.run(stream=streams[i % 2]) for i in range(8)]
    torch.cuda.synchronize()
    assert all(torch.equal(y, want) for y in got)


def test_rows_of_a_batch_do_not_depend_on_the_others(dev):
    """Appending rows keeps the bits of the first ones as long as the form of the product stays the same."""
    p = Problem(dev, 48, 300, 512, bias=F32)
    y = p.run()
    p.x = torch.cat([p.x[:37], torch.full((11, 512), float("nan"), dtype=BF16, device=dev)])
    assert torch.equal(p.run()[:37], y[:37])


@pytest.mark.parametrize("T,N,K", [(4, 256, 1024), (2000, 512, 512)])
def test_a_wait_that_runs_out(dev, T, N, K):
    p = Problem(dev, T, N, K)
    want = p.run()
    y = torch.full_like(want, 3.0)
    p.run(out=y, flags=0x100)
    assert ops.device_error() == ops.DEVERR_TIMEOUT
    # (a split product withholds the loads of a cluster's last CTA only: its whole tile stays unwritten)
    assert torch.all(y == 3.0)
    assert torch.equal(p.run(), want)
    assert ops.device_error() == 0


def test_no_tokens(dev):
    w = torch.zeros(40, 64, dtype=BF16, device=dev)
    assert ops.linear(torch.zeros(0, 64, dtype=BF16, device=dev), w).shape == (0, 40)
    assert ops.device_error() == 0


# (split over a cluster, in one run of K a CTA or more; the last two in pairs)
@pytest.mark.parametrize("T,K", [(40, 16384), (2000, 16384), (3, 40000), (16, 11200), (100, 9000), (1, 140000), (100, 70000)])
def test_long_sums_in_float32(dev, T, K):
    """An error that grows with the number of terms would show.  The tensor core cuts its sum off every 16 products, by
    half of 2**-23 of it on average, 0.72 of that over the mantissas; the sum grows as a root, which leaves 2/3: a run
    of 1024 products drifts by 64 * 2/3 * 0.72 * 2**-24 = 1.8e-6 of itself, and runs do not drift together."""
    p = Problem(dev, T, 256, K, BF16, F32)
    y = p.run()
    p.check(y)
    ref = oracle.linear.linear(wide(p.x), wide(p.w))
    assert np.linalg.norm(wide(y) - ref) <= 2e-6 * np.linalg.norm(ref)
