"""A whole MoE block, from activations and router logits to the block's output.

TEST INFRASTRUCTURE ONLY (see the package docstring).

Definition: the router choice (``oracle/gate.py``), the routed expert path with
its gate-up product, SwiGLU into the quantised operand and down product
(``quantise``, ``route``, ``gemm``, ``swiglu``), the weighted combine, and an
optional expert that every token takes, whose down product is added to the
combine's bf16 before one more rounding.  Every intermediate is rounded where
the library stores it (bf16 products, E4M3 operands).

Pins: ``tests/test_oracle_block.py`` (a token-by-token restatement without
routing, tokens that no expert takes, the always-active expert alone).
"""

import numpy as np

from . import combine, formats, gate, gemm, quantise, route, swiglu


def dense(a_q, a_sf_bytes, w_bits, addend_bits=None):
    """bf16 bits of one weight matrix's product; rows and columns of w [N, K] padded with zeros to 128."""
    w = np.pad(w_bits, ((0, -w_bits.shape[0] % 128), (0, -w_bits.shape[1] % 128)))
    bq, bsf = quantise.quantise_weight(w[None])
    d = gemm.dequant_rows(a_q, a_sf_bytes) @ gemm.dequant_weight(bq[0], bsf[0])[:w_bits.shape[0]].T
    if addend_bits is not None:
        d = d + formats.bf16_bits_to_f64(addend_bits)
    return formats.bf16_round(d)


def moe_block(x_bits, logits, w13_bits, w2_bits, kr, shared=None, **gate_args):
    """(z bf16 bits [T, K], ids [T, kr], margin [T] of the choice); ``gate_args`` as in ``gate.gate``."""
    ids, weights, margin = gate.gate(logits, kr, **gate_args)
    r = route.route(ids, w13_bits.shape[0], route.CONTIGUOUS, align=1)
    aq, asf = quantise.quantise_act(x_bits)
    rows = route.scatter_rows(aq, r["token_of_row"])
    rows_sf = route.scatter_rows(asf, r["token_of_row"], pad_value=127)
    seg, counts = r["seg_start"], r["counts"]
    y, _ = gemm.grouped_gemm(rows, rows_sf, *quantise.quantise_weight(w13_bits), seg, counts)
    y2, _ = gemm.grouped_gemm(*swiglu.swiglu_quantise(y), *quantise.quantise_weight(w2_bits), seg, counts)
    z = combine.combine(y2, r["output_index"], weights.astype(np.float32))
    if shared is not None:
        h = swiglu.swiglu_quantise(dense(aq, asf, shared[0]))
        z = dense(*h, shared[1], z)
    return z, ids, margin
