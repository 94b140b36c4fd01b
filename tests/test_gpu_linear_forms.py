"""Every form of linear's kernels by name: the sizes are looked for with ``linear_form``, so that a change of the rule that
chooses among them does not change what is covered.  Split products over 1 to 8 CTAs; pairs whose tiles come in several
rounds (the second accumulators and the hand-over between tiles) and in every width, with an epilogue of three and more
chunks a warp, with and without a residual, in words of two columns and one by one."""

import random

import pytest
import torch

from block_scaled_fp8_route_gb300 import ops
from tests.gpu_util import require_gpu
from tests.test_gpu_linear import BF16, F16, F32, Problem

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    return require_gpu()


def pairs_at_once(dev):
    return torch.cuda.get_device_properties(dev).multi_processor_count // 2


def find(seed, want, T, N, K, out, residual, odd=False):
    """Sizes of these ranges (by their logarithms) for which want(pairs, tokens, split, tiles) holds."""
    rng = random.Random(seed)
    for _ in range(100000):
        t, n, k = (int(round(lo * (hi / lo) ** rng.random())) for lo, hi in (T, N, K))
        n = n // 2 * 2 + odd
        if n > 0 and t * n * k <= 12e9 and t * n <= 12e6 and want(*ops.linear_form(t, n, k, out, residual)):
            return t, n, k
    raise AssertionError("no product of these sizes takes the form")


def run(dev, sizes, dtype, out, residual, act=None, y=None, seed=0):
    T, N, K = sizes
    p = Problem(dev, T, N, (K + 7) // 8 * 8, dtype, out, bias=F32, act=act, residual=residual, seed=seed)
    p.x, p.w = p.x[:, :K], p.w[:, :K]                    # rows strided past K
    got = p.run() if y is None else p.run(out=y)
    p.check(got)
    return p, got


@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("residual", [False, True])
# (more than 64 tokens a tile have an SM to themselves; over 1 and 7 CTAs such tiles hardly ever win)
@pytest.mark.parametrize("split,wide", [(s, False) for s in range(1, 9)] + [(s, True) for s in (2, 3, 4, 5, 6, 8)])
def test_split(dev, split, wide, residual, out):
    sizes = find(split, lambda pairs, tok, s, tiles: not pairs and s == split and (tok > 64) == wide,
                 (65, 2000) if wide else (1, 200), (8, 6000), (64, 8192), out, residual, odd=bool(split & 1))
    run(dev, sizes, BF16, out, residual, "silu", seed=split)


@pytest.mark.parametrize("dtype,residual,odd", [(BF16, False, False), (BF16, True, False), (F16, True, False), (F16, False, True),
                                                (BF16, True, True)])
@pytest.mark.parametrize("least,most,rounds", [(64, 128, 1), (144, 160, 1), (176, 192, 1), (176, 192, 2), (208, 224, 2),
                                               (240, 256, 1), (240, 256, 2)])
def test_pairs_of_several_rounds(dev, least, most, rounds, dtype, residual, odd):
    sizes = find(least + rounds, lambda pairs, tok, s, tiles: pairs and least <= tok <= most and tiles > rounds * pairs_at_once(dev),
                 (500, 9000), (256, 9000), (16, 1200), dtype, residual, odd)
    run(dev, sizes, dtype, dtype, residual, seed=least)


@pytest.mark.parametrize("residual,odd", [(False, False), (True, False), (True, True)])
@pytest.mark.parametrize("K,rounds", [((64, 1000), 2), ((1100, 2100), 2), ((3500, 5000), 1)])
def test_pairs_of_several_rounds_in_float32(dev, K, rounds, residual, odd):
    sizes = find(K[0], lambda pairs, tok, s, tiles: pairs and tok > 96 and tiles > rounds * pairs_at_once(dev), (2000, 9000),
                 (300, 3000), K, F32, residual, odd)
    run(dev, sizes, BF16, F32, residual, "sigmoid", seed=K[0])


@pytest.mark.parametrize("act", ["relu", "silu", "gelu", "gelu_tanh", "sigmoid"])
def test_pairs_with_activations(dev, act):
    sizes = find(len(act), lambda pairs, tok, s, tiles: pairs and tok > 160 and tiles > pairs_at_once(dev), (1500, 4000),
                 (600, 2000), (64, 600), F16, True)
    run(dev, sizes, F16, F16, True, act)


@pytest.mark.parametrize("out", [BF16, F16])
def test_pairs_onto_the_residual_and_between_other_values(dev, out):
    """y is the residual, inside a buffer that keeps what is around it, aligned to four, two and one values."""
    T, N, K = find(3, lambda pairs, tok, s, tiles: pairs and tok > 160 and tiles > pairs_at_once(dev), (2000, 4000), (1000, 3000),
                   (64, 600), out, True)
    p, want = run(dev, (T, N, K), out, out, True)
    for left, pitch in ((0, N + 8), (2, N + 6), (1, N + 4), (2, N + 5)):
        buf = torch.full((T + 2, pitch), 7.0, dtype=out, device=dev)
        y = buf[1:1 + T, left:left + N]
        y.copy_(p.residual)
        p.run(out=y, residual=y)
        assert torch.equal(y, want)
        y.fill_(7.0)
        assert torch.all(buf == 7.0)


def test_pairs_of_several_rounds_in_a_graph_and_back_to_back(dev):
    n = pairs_at_once(dev)
    a = find(5, lambda pairs, tok, s, tiles: pairs and tok > 192 and tiles > 2 * n, (2000, 9000), (1000, 3000), (64, 600), BF16, True)
    b = find(6, lambda pairs, tok, s, tiles: pairs and tok <= 128 and tiles > n, (500, 9000), (256, 9000), (200, 1200), BF16, False)
    cases = [run(dev, a, BF16, BF16, True), run(dev, b, BF16, BF16, False, "gelu")]
    graph, outs = torch.cuda.CUDAGraph(), [torch.empty_like(want) for _, want in cases]
    with torch.cuda.graph(graph):
        for _ in range(3):
            for (p, _), y in zip(cases, outs):
                p.run(out=y)
    for y in outs:
        y.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(y, want) for y, (_, want) in zip(outs, cases))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [cases[i % 2][0].run(stream=streams[i % 2]) for i in range(8)]
    torch.cuda.synchronize()
    assert all(torch.equal(y, cases[i % 2][1]) for i, y in enumerate(got))


def test_a_wait_that_runs_out_ends_all_rounds(dev):
    sizes = find(7, lambda pairs, tok, s, tiles: pairs and tok > 160 and tiles > pairs_at_once(dev), (1500, 4000), (600, 2000),
                 (64, 600), BF16, False)
    p, want = run(dev, sizes, BF16, BF16, False)
    y = torch.full_like(want, 3.0)
    p.run(out=y, flags=0x100)
    assert ops.device_error() == ops.DEVERR_TIMEOUT
    assert torch.all(y == 3.0)
    assert torch.equal(p.run(), want) and ops.device_error() == 0
