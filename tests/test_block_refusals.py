"""Refusals of gate, swiglu_quantise and dense_gemm: every host-side check returns its documented
status, and the binding refuses wrong types, shapes and host tensors, before any device call."""

import ctypes

import pytest
import torch

from block_scaled_fp8_route_gb300 import _lib, build, ops

INVALID, MISALIGNED, UNSUPPORTED = 1, 2, 3
NUL, OK, ODD = ctypes.c_void_p(0), ctypes.c_void_p(256), ctypes.c_void_p(257)


@pytest.fixture(scope="module")
def lib():
    return _lib.load(build.build())


def test_gate(lib):
    def gate(logits=OK, kind=0, T=4, E=64, ld=64, bias=NUL, groups=1, kept=1, kr=8, flags=0, scale=1.0, ids=OK, w=OK):
        return lib.bsf_gate(logits, kind, T, E, ld, bias, groups, kept, kr, flags, scale, ids, w, NUL)
    assert gate(T=0) == 0
    for bad in (dict(T=-1), dict(E=0), dict(kr=0), dict(groups=0), dict(kept=0), dict(kind=2), dict(flags=8),
                dict(groups=65), dict(groups=5), dict(kept=2), dict(kr=65), dict(ld=63),
                dict(groups=8, kept=2, kr=17), dict(scale=float("nan")), dict(scale=float("inf")),
                dict(logits=NUL), dict(ids=NUL), dict(w=NUL)):
        assert gate(**bad) == INVALID, bad
    for bad in (dict(E=1025, ld=1025), dict(E=64, groups=64, kept=64), dict(kr=33), dict(T=2**40),
                dict(ld=2**25)):
        assert gate(**bad) == UNSUPPORTED, bad
    for bad in (dict(logits=ODD), dict(logits=ctypes.c_void_p(258)), dict(bias=ODD), dict(ids=ODD), dict(w=ODD)):
        assert gate(**bad) == MISALIGNED, bad


def test_swiglu_quantise(lib):
    def swiglu(y=OK, T=4, K=128, ld=256, tok=NUL, used=NUL, q=OK, sf=OK, sf_ld=4):
        return lib.bsf_swiglu_quantise(y, T, K, ld, tok, used, q, sf, sf_ld, NUL)
    assert swiglu(T=0) == 0
    for bad in (dict(T=-1), dict(K=0), dict(K=12), dict(ld=255), dict(y=NUL), dict(q=NUL), dict(sf=NUL), dict(tok=OK),
                dict(used=OK), dict(sf_ld=3), dict(T=5), dict(sf_ld=6)):
        assert swiglu(**bad) == INVALID, bad
    for bad in (dict(y=ODD), dict(q=ODD), dict(sf=ODD), dict(ld=260)):
        assert swiglu(**bad) == MISALIGNED, bad
    assert swiglu(T=2**40, sf_ld=2**40) == UNSUPPORTED
    assert swiglu(ld=2**25) == UNSUPPORTED


def test_dense_gemm(lib):
    def dense(a=OK, sfa=OK, sfa_ld=8, M=8, b=OK, sfb=OK, N=200, K=256, c=NUL, ldc=0, d=OK, ldd=200, flags=2):
        return lib.bsf_dense_gemm(a, sfa, sfa_ld, M, b, sfb, N, K, c, ldc, d, ldd, flags, NUL)
    assert dense(M=0) == 0
    for bad in (dict(M=-1), dict(N=0), dict(K=0), dict(K=200), dict(flags=1), dict(flags=4), dict(a=NUL),
                dict(sfa=NUL), dict(b=NUL), dict(sfb=NUL), dict(d=NUL), dict(sfa_ld=4), dict(sfa_ld=9),
                dict(ldd=199), dict(c=OK, ldc=199)):
        assert dense(**bad) == INVALID, bad
    for bad in (dict(a=ODD), dict(b=ODD), dict(sfa=ODD), dict(sfb=ODD), dict(d=ODD), dict(c=ODD, ldc=200)):
        assert dense(**bad) == MISALIGNED, bad
    for bad in (dict(M=2**40, sfa_ld=2**40), dict(N=2**25, ldd=2**25), dict(K=2**25), dict(ldd=2**25),
                dict(c=OK, ldc=2**25), dict(N=2**23, ldd=2**23, K=2**20)):
        assert dense(**bad) == UNSUPPORTED, bad


def test_binding_refuses_what_a_kernel_would_misread():
    f, h = torch.zeros(4, 64), torch.zeros(4, 64, dtype=torch.float16)
    with pytest.raises(ValueError, match="CUDA tensor"):
        ops.gate(f, 2)
    with pytest.raises(ValueError, match="float32 or bfloat16"):
        ops.gate(h, 2)
    with pytest.raises(ValueError, match="softmax or sigmoid"):
        ops.gate(f, 2, score="relu")
    with pytest.raises(ValueError, match="contiguous rows"):
        ops.gate(f.t(), 2)
    with pytest.raises(ValueError, match="topk_ids"):
        ops.gate(f, 2, topk_ids=torch.zeros(4, 3, dtype=torch.int32))
    with pytest.raises(ValueError, match="bias"):
        ops.gate(f, 2, bias=torch.zeros(63))

    y = torch.zeros(4, 256, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA tensor"):
        ops.swiglu_quantise(y)
    with pytest.raises(ValueError, match="bfloat16"):
        ops.swiglu_quantise(y.float())
    with pytest.raises(ValueError, match="even number"):
        ops.swiglu_quantise(y[:, :255])
    with pytest.raises(ValueError, match="q:"):
        ops.swiglu_quantise(y, q=torch.zeros(4, 64, dtype=torch.uint8))
    with pytest.raises(ValueError, match="rows"):
        ops.swiglu_quantise(y, rows=(torch.zeros(3, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)))

    a, sfa = torch.zeros(4, 128, dtype=torch.uint8), torch.zeros(1, 4, dtype=torch.int32)
    b, sfb = torch.zeros(256, 128, dtype=torch.uint8), torch.zeros(1, 256, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA tensor"):
        ops.dense_gemm(a, sfa, b, sfb)
    with pytest.raises(ValueError, match="rows for N"):
        ops.dense_gemm(a, sfa, b, sfb, 128)
    with pytest.raises(ValueError, match="sfb"):
        ops.dense_gemm(a, sfa, b, sfb[:, :128], 256)
    with pytest.raises(ValueError, match="addend"):
        ops.dense_gemm(a, sfa, b, sfb, 200, addend=torch.zeros(4, 100, dtype=torch.bfloat16, device="meta"))
    with pytest.raises(ValueError, match="d:"):
        ops.dense_gemm(a, sfa, b, sfb, 200, d=torch.zeros(4, 256, dtype=torch.bfloat16))
