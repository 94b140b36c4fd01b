"""Refusals of few_token_moe and linear: every host-side check returns its documented status, and the binding refuses
wrong types, shapes, devices and streams, before any device call.  CPU-only."""

import ctypes

import pytest
import torch

from block_scaled_fp8_route_gb300 import MoEBlock, MoEPath, _lib, build, ops

INVALID, MISALIGNED, UNSUPPORTED = 1, 2, 3
NUL, OK, ODD = ctypes.c_void_p(0), ctypes.c_void_p(256), ctypes.c_void_p(257)
F32, F16, BF16, I32, U8 = torch.float32, torch.float16, torch.bfloat16, torch.int32, torch.uint8


@pytest.fixture(scope="module")
def lib():
    return _lib.load(build.build())


def few(lib, x=OK, T=4, K=256, ldx=256, ids=OK, p=OK, kr=2, E=8, I=128, kind=2, w13=OK, f13=OK, w2=OK, f2=OK, S=0,
        s13=NUL, sf13=NUL, s2=NUL, sf2=NUL, c=NUL, ldc=0, z=OK, ldz=256, ws=OK, size=1 << 40, flags=2):
    return lib.bsf_few_token_moe(x, T, K, ldx, ids, p, kr, E, I, kind, w13, f13, w2, f2, S, s13, sf13, s2, sf2, c, ldc,
                                 z, ldz, ws, size, flags, NUL)


def test_few_token_moe_statuses(lib):
    shared = dict(S=128, s13=OK, sf13=OK, s2=OK, sf2=OK)
    assert few(lib, T=0) == 0 and few(lib, T=0, **shared) == 0
    for bad in (dict(T=-1), dict(K=0), dict(kr=0), dict(E=0), dict(I=0), dict(S=-128), dict(K=200), dict(I=100),
                dict(S=64), dict(kind=0), dict(kind=3), dict(flags=1), dict(flags=4), dict(x=NUL), dict(ids=NUL),
                dict(p=NUL), dict(w13=NUL), dict(w2=NUL), dict(z=NUL), dict(ws=NUL), dict(f13=NUL), dict(f2=NUL),
                dict(ldx=248), dict(ldz=255), dict(c=OK, ldc=255), dict(size=1000)):
        assert few(lib, **bad) == INVALID, bad
    for name in ("s13", "sf13", "s2", "sf2"):
        assert few(lib, **{**shared, name: NUL}) == INVALID, name
    for bad in (dict(T=33), dict(kr=33), dict(E=1025), dict(K=2**23 + 128, ldx=2**23 + 128, ldz=2**23 + 128),
                dict(I=2**25), dict(S=2**25), dict(ldx=2**25), dict(ldz=2**25), dict(c=OK, ldc=2**25),
                dict(E=1024, I=2**20, K=2**20, ldx=2**20, ldz=2**20)):
        assert few(lib, **bad) == UNSUPPORTED, bad
    for bad in (dict(x=ODD), dict(ldx=260), dict(w13=ODD), dict(w2=ODD), dict(ws=ODD), dict(ids=ODD), dict(p=ODD),
                dict(f13=ODD), dict(f2=ODD), dict(z=ODD), dict(c=ODD, ldc=256), {**shared, "s13": ODD},
                {**shared, "s2": ODD}, {**shared, "sf13": ODD}, {**shared, "sf2": ODD}):
        assert few(lib, **bad) == MISALIGNED, bad


def test_few_token_moe_workspace(lib):
    size = lib.bsf_few_token_moe_workspace_bytes
    assert size(4, 2, 128, 0) >= 4 * 8 * 2 * 128 * 4               # four float32 sums of gate and up of every row
    assert size(4, 2, 128, 256) >= size(4, 2, 128, 0) + 4 * 4 * 2 * 256 * 4
    for bad in ((33, 2, 128, 0), (4, 33, 128, 0), (-1, 2, 128, 0), (4, 0, 128, 0), (4, 2, 0, 0), (4, 2, 2**40, 0),
                (4, 2, 128, -1), (4, 2, 128, 2**40)):
        assert size(*bad) == 0
        with pytest.raises(ValueError, match="few_token_moe"):
            ops.few_token_moe_workspace(*bad)
    need = size(4, 2, 128, 0)
    assert few(lib, size=need - 1) == INVALID


def lin(lib, x=OK, kind=1, T=4, K=100, ldx=104, w=OK, N=60, ldw=104, b=NUL, bk=0, act=0, r=NUL, ldr=0, y=OK, yk=1,
        ldy=60, flags=0):
    return lib.bsf_linear(x, kind, T, K, ldx, w, N, ldw, b, bk, act, r, ldr, y, yk, ldy, flags, NUL)


def test_linear_statuses(lib):
    assert lin(lib, T=0) == 0
    for bad in (dict(T=-1), dict(N=0), dict(K=0), dict(kind=0), dict(kind=2), dict(kind=4), dict(yk=2), dict(yk=4),
                dict(b=OK, bk=2), dict(act=-1), dict(act=6), dict(flags=1), dict(flags=2), dict(x=NUL), dict(w=NUL),
                dict(y=NUL), dict(ldx=96), dict(ldw=96), dict(ldy=59), dict(r=OK, ldr=59)):
        assert lin(lib, **bad) == INVALID, bad
    for bad in (dict(x=ODD), dict(w=ODD), dict(ldx=108), dict(ldw=108), dict(y=ODD), dict(r=ODD, ldr=60),
                dict(b=ODD, bk=1), dict(b=ctypes.c_void_p(258), bk=0), dict(y=ctypes.c_void_p(258), yk=0),
                dict(r=ctypes.c_void_p(258), ldr=60, yk=0), dict(x=ctypes.c_void_p(264)), dict(w=ctypes.c_void_p(264))):
        assert lin(lib, **bad) == MISALIGNED, bad
    for bad in (dict(T=2**40), dict(T=2**31 - 100), dict(N=2**25, ldy=2**25), dict(K=2**25, ldx=2**25, ldw=2**25),
                dict(ldx=2**25), dict(ldw=2**25), dict(ldy=2**25), dict(r=OK, ldr=2**25)):
        assert lin(lib, **bad) == UNSUPPORTED, bad


def test_python_constants_match_the_header():
    import os
    import re
    with open(os.path.join(build.ROOT, "include", "bsfroute.h"), encoding="utf-8") as f:
        defs = dict(re.findall(r"#define BSF_(\w+) (\d+)", f.read()))
    assert ops.TYPE_E4M3 == int(defs["TYPE_E4M3"])
    assert ops._LINEAR_TYPES == {F32: int(defs["TYPE_F32"]), BF16: int(defs["TYPE_BF16"]), F16: int(defs["TYPE_F16"])}
    assert ops._ACTIVATIONS == {None: 0, **{k.lower(): int(defs["ACT_" + k]) for k in
                                            ("NONE", "RELU", "SILU", "GELU", "GELU_TANH", "SIGMOID")}}


class Reached(Exception):
    pass


class Tensor:
    """What the binding asks of a CUDA tensor."""
    is_cuda = True

    def __init__(self, *shape, dtype, device=0, stride=None):
        self._meta = torch.empty(shape, dtype=dtype, device="meta") if stride is None else \
            torch.empty_strided(shape, stride, dtype=dtype, device="meta")
        self.dtype, self.shape, self.device, self._index = dtype, self._meta.shape, f"cuda:{device}", device

    def get_device(self):
        return self._index

    def __getattr__(self, name):
        if name in ("dim", "stride", "is_contiguous", "numel"):
            return getattr(self._meta, name)
        raise AttributeError(name)

    def data_ptr(self):
        return 256

    def record_stream(self, stream):
        pass


class Stream:
    cuda_stream = 0

    def __init__(self, device):
        self.device_index = device


class Library:
    """Stands for the library: sizes as it would give them, and no launch."""

    @staticmethod
    def bsf_few_token_moe_workspace_bytes(T, kr, I, S):
        return 4096

    @staticmethod
    def bsf_few_token_moe(*a):
        raise Reached

    bsf_linear = bsf_few_token_moe


@pytest.fixture
def library(monkeypatch):
    monkeypatch.setattr(_lib, "load", lambda: Library)
    monkeypatch.setattr(ops, "_current_device", lambda: 0, raising=False)
    monkeypatch.setattr(ops, "_current_stream", lambda device: 0)


def moe_operands(kind=U8, dev=None, **other):
    wide = 2 if kind == BF16 else 1
    shapes = dict(x=((4, 256), BF16), topk_ids=((4, 2), I32), topk_weights=((4, 2), F32), w13=((8, 256, 256 * wide), U8),
                  sfb13=((8, 1, 256), I32), w2=((8, 256, 128 * wide), U8), sfb2=((8, 1, 256), I32),
                  shared_w13=((512, 256 * wide), U8), shared_sfb13=((1, 512), I32), shared_w2=((256, 256 * wide), U8),
                  shared_sfb2=((1, 256), I32), addend=((4, 256), BF16), z=((4, 256), BF16), workspace=((4096,), U8))
    t = {k: Tensor(*s, dtype=d, device=(dev or {}).get(k, 0)) for k, (s, d) in shapes.items()}
    if kind == BF16:
        t.update(sfb13=None, sfb2=None, shared_sfb13=None, shared_sfb2=None)
    t.update(other)
    return t


def moe(t, stream=None):
    shared = tuple(t["shared_" + k] for k in ("w13", "sfb13", "w2", "sfb2"))
    return ops.few_token_moe(t["x"], t["topk_ids"], t["topk_weights"], t["w13"], t["sfb13"], t["w2"], t["sfb2"],
                             shared=None if shared[0] is None else shared, addend=t["addend"], z=t["z"],
                             workspace=t["workspace"], stream=stream)


def test_few_token_moe_takes_matching_operands(library):
    for kind in (U8, BF16):
        for stream in (None, Stream(0)):
            with pytest.raises(Reached):
                moe(moe_operands(kind), stream)
    plain = moe_operands(BF16, w13=Tensor(8, 256, 256, dtype=BF16), w2=Tensor(8, 256, 128, dtype=BF16),
                         shared_w13=Tensor(512, 256, dtype=BF16), shared_w2=Tensor(256, 256, dtype=BF16))
    with pytest.raises(Reached):
        moe(plain)


@pytest.mark.parametrize("name", [k for k in moe_operands()])
def test_few_token_moe_operands_on_another_device(library, name):
    with pytest.raises(ValueError, match=f"{name} on cuda:1"):
        moe(moe_operands(dev={name: 1}))
    with pytest.raises(ValueError, match="stream on cuda:1"):
        moe(moe_operands(), Stream(1))


@pytest.mark.parametrize("other", [
    dict(x=Tensor(4, 256, dtype=F16)), dict(x=Tensor(4, 2, 128, dtype=BF16)),
    dict(x=Tensor(4, 256, dtype=BF16, stride=(1, 4))), dict(topk_ids=Tensor(4, 2, dtype=torch.int64)),
    dict(topk_ids=Tensor(3, 2, dtype=I32)), dict(topk_weights=Tensor(4, 3, dtype=F32)),
    dict(topk_weights=Tensor(4, 2, dtype=BF16)), dict(topk_ids=Tensor(4, 2, dtype=I32, stride=(1, 4))),
    dict(w13=Tensor(8, 256, 128, dtype=U8)), dict(w13=Tensor(256, 256, dtype=U8)), dict(w13=Tensor(8, 256, 256, dtype=I32)),
    dict(w2=Tensor(8, 128, 128, dtype=U8)), dict(w2=Tensor(7, 256, 128, dtype=U8)),
    dict(sfb13=Tensor(8, 2, 256, dtype=I32)), dict(sfb13=Tensor(8, 1, 256, dtype=F32)), dict(sfb2=None),
    dict(shared_w13=Tensor(8, 512, 256, dtype=U8)), dict(shared_w2=Tensor(256, 128, dtype=U8)),
    dict(shared_sfb13=None), dict(shared_sfb2=Tensor(2, 256, dtype=I32)), dict(addend=Tensor(4, 256, dtype=F32)),
    dict(addend=Tensor(5, 256, dtype=BF16)), dict(z=Tensor(4, 128, dtype=BF16)), dict(z=Tensor(4, 256, dtype=F32)),
    dict(z=Tensor(4, 256, dtype=BF16, stride=(1, 4))), dict(workspace=Tensor(4095, dtype=U8)),
    dict(workspace=Tensor(4096, dtype=F32))])
def test_few_token_moe_refuses_other_operands(library, other):
    with pytest.raises(ValueError):
        moe(moe_operands(**other))


@pytest.mark.parametrize("name", ["x", "z", "addend"])
def test_few_token_moe_refuses_a_single_row_whose_values_are_apart(library, name):
    one = dict(x=Tensor(1, 256, dtype=BF16), topk_ids=Tensor(1, 2, dtype=I32), topk_weights=Tensor(1, 2, dtype=F32),
               addend=Tensor(1, 256, dtype=BF16), z=Tensor(1, 256, dtype=BF16))
    with pytest.raises(Reached):
        moe(moe_operands(**one))
    for stride in ((512, 2), (0, 0), (1, 1024)):
        with pytest.raises(ValueError, match=name):
            moe(moe_operands(**{**one, name: Tensor(1, 256, dtype=BF16, stride=stride)}))
    with pytest.raises(Reached):                     # (the stride between rows of a single row is not looked at)
        moe(moe_operands(**{**one, name: Tensor(1, 256, dtype=BF16, stride=(3, 1))}))


def test_few_token_moe_refuses_scales_of_bf16_weights_and_odd_sizes(library):
    with pytest.raises(ValueError, match="no scale words"):
        moe(moe_operands(BF16, sfb2=Tensor(8, 1, 256, dtype=I32)))
    t = moe_operands(w13=Tensor(8, 200, 256, dtype=U8), sfb13=Tensor(8, 1, 200, dtype=I32),
                     w2=Tensor(8, 256, 100, dtype=U8), shared_w13=None)
    with pytest.raises(ValueError, match="multiples of 128"):
        moe(t)


def lin_operands(dev=None, **other):
    shapes = dict(x=((4, 104), BF16), w=((60, 104), BF16), bias=((60,), F32), residual=((4, 60), BF16), out=((4, 60), BF16))
    t = {k: Tensor(*s, dtype=d, device=(dev or {}).get(k, 0)) for k, (s, d) in shapes.items()}
    t.update(other)
    return t


def run_linear(t, stream=None, **kw):
    return ops.linear(t["x"], t["w"], bias=t["bias"], residual=t["residual"], out=t["out"], stream=stream, **kw)


def test_linear_takes_matching_operands(library):
    for act in (None, "none", "relu", "silu", "gelu", "gelu_tanh", "sigmoid"):
        with pytest.raises(Reached):
            run_linear(lin_operands(), activation=act)
    with pytest.raises(Reached):
        run_linear(lin_operands(), Stream(0))


@pytest.mark.parametrize("name", [k for k in lin_operands()])
def test_linear_operands_on_another_device(library, name):
    with pytest.raises(ValueError, match=f"{name} on cuda:1"):
        run_linear(lin_operands({name: 1}))
    with pytest.raises(ValueError, match="stream on cuda:1"):
        run_linear(lin_operands(), Stream(1))


@pytest.mark.parametrize("other,kw", [
    (dict(x=Tensor(4, 104, dtype=F32)), {}), (dict(x=Tensor(4, 104, dtype=F16)), {}),
    (dict(x=Tensor(104, dtype=BF16)), {}), (dict(w=Tensor(60, 96, dtype=BF16)), {}),
    (dict(x=Tensor(4, 104, dtype=BF16, stride=(1, 4))), {}), (dict(w=Tensor(60, 104, dtype=BF16, stride=(1, 60))), {}),
    (dict(bias=Tensor(61, dtype=F32)), {}), (dict(bias=Tensor(60, dtype=torch.float64)), {}),
    (dict(bias=Tensor(60, dtype=F32, stride=(2,))), {}), (dict(residual=Tensor(4, 60, dtype=F32)), {}),
    (dict(residual=Tensor(3, 60, dtype=BF16)), {}), (dict(out=Tensor(4, 61, dtype=BF16)), {}),
    (dict(out=Tensor(4, 60, dtype=torch.float64)), {}), (dict(out=Tensor(4, 60, dtype=BF16, stride=(1, 4))), {}),
    ({}, dict(activation="tanh")), ({}, dict(out_dtype=F32)), ({}, dict(out_dtype=torch.int32))])
def test_linear_refuses_other_operands(library, other, kw):
    with pytest.raises(ValueError):
        run_linear(lin_operands(**other), **kw)


def test_host_tensors_are_refused():
    h = lambda *s, dtype=BF16: torch.zeros(s, dtype=dtype)  # noqa: E731
    with pytest.raises(ValueError, match="x: expected a CUDA tensor"):
        ops.linear(h(4, 64), h(8, 64))
    with pytest.raises(ValueError, match="x: expected a CUDA tensor"):
        ops.few_token_moe(h(4, 128), h(4, 2, dtype=I32), h(4, 2, dtype=F32), h(2, 256, 128), None, h(2, 128, 128), None)


@pytest.fixture
def no_quantisation(monkeypatch):
    def reached(*a, **k):
        raise Reached
    monkeypatch.setattr(ops, "quantise_weight", reached)
    monkeypatch.setattr(MoEPath, "__init__", reached)
    monkeypatch.setattr(ops, "gate", lambda *a, **k: None)


def test_block_arguments(no_quantisation):
    E, K, I = 8, 256, 128
    w = torch.zeros(E, 2 * I, K, dtype=BF16), torch.zeros(E, K, I, dtype=BF16)
    make = lambda T=4, **kw: MoEBlock(E, 2, T, K, I, *w, device="cpu", **kw)  # noqa: E731
    router, bias = torch.zeros(E, K, dtype=BF16), torch.zeros(E)
    for kw in (dict(few_tokens=True), dict(few_tokens=True, T=32), dict(router=router), dict(router=(router, bias))):
        with pytest.raises(Reached):
            make(**kw)
    with pytest.raises(ValueError, match="few_tokens"):
        make(T=33, few_tokens=True)
    for bad in (router.float(), router[:4], router[:, :128], (router, bias.to(BF16)), (router, bias[:4])):
        with pytest.raises(ValueError, match="router"):
            make(router=bad)


def test_block_steps():
    b = object.__new__(MoEBlock)
    b.T, b.K, b.E, b.kr, b.gate_args, b.few_tokens, b.router = 4, 256, 8, 2, {}, True, None
    b.z = torch.zeros(4, 256, dtype=BF16)
    x = torch.zeros(4, 256, dtype=BF16)
    with pytest.raises(ValueError, match="no router"):
        b.step(x)
    with pytest.raises(ValueError, match="logits"):
        b.step(x, torch.zeros(4, 9))
    with pytest.raises(ValueError, match="addend"):
        b.step(x, torch.zeros(4, 8), addend=torch.zeros(4, 256))
    b.few_tokens, b.path = False, type("P", (), {"E": 8})
    with pytest.raises(ValueError, match="addend"):
        b.step(x, torch.zeros(4, 8), addend=x)
