"""How exactly ``few_token_moe`` carries h into its second product: within the bound of three E4M3 terms, or of two bf16
terms, alone and over the sizes at which operands, accumulators and scales change places."""

import numpy as np
import pytest
import torch

import oracle
from block_scaled_fp8_route_gb300 import ops
from tests.few_cases import cancelling
from tests.gpu_util import require_gpu
from tests.test_gpu_few_tokens import Layer, f64, inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    return require_gpu()


class TermsLayer(Layer):
    """The same checks, with the bound of the terms that h is split into."""

    def check(self, z, x, ids, p, addend=None):
        assert ops.device_error() == 0
        args = (f64(x), ids.cpu().numpy(), p.cpu().numpy(), self.wide13, self.wide2, self.wide_shared,
                None if addend is None else f64(addend))
        ref = oracle.few_tokens.few_token_moe(*args)
        tol = oracle.few_tokens.bound(*args, fp8=self.fp8, terms=3 if self.fp8 else 2)
        tol = tol + 2.0 ** -8 * (np.abs(ref) + tol)
        worst = np.max(np.abs(f64(z) - ref) / tol)
        assert worst <= 1, f"worst {worst:.2f} times the bound"


@pytest.mark.parametrize("fmt", ["fp8", "bf16"])
@pytest.mark.parametrize("T", [1, 3, 8, 9, 17, 24, 25, 32])
def test_errors_of_single_values(dev, fmt, T):
    for seed in range(3):
        host = cancelling(T, seed=seed)
        x, ids, p, w13, w2 = (t.to(dev) for t in host)
        if fmt == "fp8":
            def made(w):
                q, sf128 = ops.quantise_weight(w)
                bq, bsf = oracle.quantise.quantise_weight(w.cpu().view(torch.int16).numpy().view(np.uint16))
                assert np.array_equal(np.stack([oracle.gemm.dequant_weight(bq[e], bsf[e]) for e in range(len(bq))]), f64(w))
                return ops.tile_weights(q), ops.prepare_weight_sf(sf128, w.shape[2])
            (b13, f13), (b2, f2) = made(w13), made(w2)
        else:
            b13, f13, b2, f2 = ops.tile_weights(w13), None, ops.tile_weights(w2), None
        z = ops.few_token_moe(x, ids, p, b13, f13, b2, f2)
        assert ops.device_error() == 0
        args = [f64(t) if t.dtype == torch.bfloat16 else t.numpy() for t in host]
        tol = oracle.few_tokens.bound(*args, fp8=fmt == "fp8", terms=3 if fmt == "fp8" else 2)
        ref = oracle.few_tokens.few_token_moe(*args)
        worst = np.max(np.abs(f64(z) - ref) / (tol + 2.0 ** -8 * (np.abs(ref) + tol)))
        assert worst <= 1, f"worst {worst:.2f} times the bound"


@pytest.mark.parametrize("fmt", ["fp8", "bf16"])
@pytest.mark.parametrize("E,kr,K,I,S", [(1, 1, 128, 128, 0), (2, 1, 128, 640, 0), (33, 5, 640, 384, 128), (16, 16, 384, 256, 0),
                                        (40, 3, 2048, 128, 512), (6, 2, 2176, 128, 0), (4, 2, 1920, 640, 0)])
def test_sizes(dev, fmt, E, kr, K, I, S):
    layer = TermsLayer(dev, E, K, I, S, fmt=fmt, seed=E)
    for T in (1, 7, 8, 16, 17, 31, 32):
        x, ids, p = inputs(dev, T, K, E, kr, T)
        if T > 8:
            ids[1] = -1
        layer.check(layer.call(x, ids, p), x, ids, p)


def test_values_far_apart_in_a_block(dev):
    layer = TermsLayer(dev, 4, 256, 128)
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
@pytest.mark.parametrize("T", [1, 9, 16, 17, 32])
def test_every_block_of_weights_has_an_exponent_of_its_own(dev, fmt, T):
    """Neighbouring tiles of a CTA (gate and up rows; two tiles of w2) meet one operand with different scales."""
    E, K, I, S = 5, 1536, 384, 256
    layer = TermsLayer(dev, E, K, I, S, fmt=fmt)
    g = torch.Generator().manual_seed(T)

    def made(n, rows, inner):
        w = torch.randn(n, rows // 128, 128, inner // 128, 128, generator=g) * 0.05
        w *= torch.exp2(torch.randint(-4, 5, (n, rows // 128, 1, inner // 128, 1), generator=g).float())
        w = w.view(n, rows, inner).to(torch.bfloat16).to(dev)
        if fmt == "bf16":
            return ops.tile_weights(w), None, f64(w)
        q, sf128 = ops.quantise_weight(w)
        bq, bsf = oracle.quantise.quantise_weight(w.cpu().view(torch.int16).numpy().view(np.uint16))
        assert len(np.unique(bsf)) > 4
        return ops.tile_weights(q), ops.prepare_weight_sf(sf128, inner), np.stack(
            [oracle.gemm.dequant_weight(bq[e], bsf[e]) for e in range(n)])

    layer.w13, layer.sf13, layer.wide13 = made(E, 2 * I, K)
    layer.w2, layer.sf2, layer.wide2 = made(E, K, I)
    a, b = made(1, 2 * S, K), made(1, K, S)
    layer.shared = tuple(None if t is None else t[0] for t in (a[0], a[1], b[0], b[1]))
    layer.wide_shared = (a[2][0], b[2][0])
    x, ids, p = inputs(dev, T, K, E, 2, T)
    layer.check(layer.call(x, ids, p), x, ids, p)
