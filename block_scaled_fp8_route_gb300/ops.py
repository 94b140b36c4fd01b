"""Thin torch-facing binding of the C ABI (argument marshalling only).

Every function here allocates its outputs with torch (device memory is the
only thing torch provides), passes raw pointers and the current CUDA stream to
``libbsfroute.so`` and returns the tensors.  All arithmetic runs in the CUDA
kernels.  Names follow the C entry points without the ``bsf_`` prefix.
"""

import ctypes

import torch

from . import _lib

CONTIGUOUS = 0
MASKED = 1
B_HOST_MAPPED = 1
B_TILED = 2              # weights in the layout of tile_weights()
# device error bits (BSF_DEVERR_* in bsfroute.h), read with device_error()
DEVERR_EXPERT_ID = 0x1
DEVERR_MASKED_OVERFLOW = 0x2
DEVERR_TIMEOUT = 0x4
DEVERR_BAD_SCALE = 0x8
DEVERR_SEGMENT = 0x10


def _ptr(t):
    """Device pointer of a CUDA tensor; a host tensor here would be read or written by a kernel
    through an address it cannot use, so it is refused before any library call."""
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError(f"expected a CUDA tensor, got one on {t.device}")
    return ctypes.c_void_p(t.data_ptr())


def _wptr(t, flags):
    """Weights / weight scales: CUDA tensors, or pinned host tensors with B_HOST_MAPPED."""
    if t is None:
        return None
    if flags & B_HOST_MAPPED:
        if t.is_cuda or not t.is_pinned():
            raise ValueError("B_HOST_MAPPED weights must be pinned host tensors (tensor.pin_memory())")
        return ctypes.c_void_p(t.data_ptr())
    return _ptr(t)


def _stream(stream=None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def sf_ld(rows: int) -> int:
    """Row stride (int32 words) of a packed MN-major SF tensor: rows rounded up to 4."""
    return (rows + 3) // 4 * 4


def sf_words(K: int) -> int:
    return (K // 128 + 3) // 4


def device_error(clear: bool = True, stream=None) -> int:
    code = ctypes.c_int32(0)
    _lib.check(_lib.load().bsf_get_device_error(ctypes.byref(code), int(clear), _stream(stream)), "get_device_error")
    return code.value


def quantise_act(x, q=None, sf=None, stream=None, rows=None):
    """x bf16 [T, K] -> (q uint8 [T, K], sf int32 [ceil(K/512), sf_ld(T)]).  ``rows`` = (token_of_row,
    rows_used) of a packed operand (a RouteBuffers' token_of_row and seg_start[E:]): only its routed
    rows are quantised, the padding rows of q and sf are left unwritten."""
    T, K = x.shape
    x = x.contiguous()
    if q is None:
        q = torch.empty((T, K), dtype=torch.uint8, device=x.device)
    if sf is None:
        sf = torch.empty((sf_words(K), sf_ld(T)), dtype=torch.int32, device=x.device)
    lib = _lib.load()
    if rows is None:
        _lib.check(lib.bsf_quantise_act(_ptr(x), T, K, _ptr(q), _ptr(sf), sf.shape[1], _stream(stream)),
                   "quantise_act")
    else:
        token_of_row, rows_used = rows
        assert token_of_row.dtype == torch.int32 and token_of_row.numel() >= T and rows_used.dtype == torch.int32
        _lib.check(lib.bsf_quantise_act_rows(_ptr(x), T, K, _ptr(token_of_row), _ptr(rows_used), _ptr(q), _ptr(sf),
                                             sf.shape[1], _stream(stream)), "quantise_act_rows")
    return q, sf


def quantise_weight(w, stream=None):
    """w bf16 [E, N, K] -> (q uint8 [E, N, K], sf128 float32 [E, N/128, K/128])."""
    E, N, K = w.shape
    w = w.contiguous()
    q = torch.empty((E, N, K), dtype=torch.uint8, device=w.device)
    sf128 = torch.empty((E, N // 128, K // 128), dtype=torch.float32, device=w.device)
    _lib.check(_lib.load().bsf_quantise_weight(_ptr(w), E, N, K, _ptr(q), _ptr(sf128), _stream(stream)),
               "quantise_weight")
    return q, sf128


def prepare_weight_sf(sf128, K: int, stream=None):
    """sf128 float32 [E, N/128, K/128] -> per-row packed int32 [E, ceil(K/512), N]."""
    E, nb, _ = sf128.shape
    N = nb * 128
    sfb = torch.empty((E, sf_words(K), N), dtype=torch.int32, device=sf128.device)
    _lib.check(_lib.load().bsf_prepare_weight_sf(_ptr(sf128.contiguous()), E, N, K, _ptr(sfb), _stream(stream)),
               "prepare_weight_sf")
    return sfb


def tile_weights(b, stream=None):
    """Weights [E, N, ...] (any dtype; rows of ``row_bytes`` bytes) -> the same bytes tiled
    [E][N/128][row_bytes/128][128][128] for the GEMM flag ``B_TILED``; returned as uint8
    [E, N, row_bytes] so that its shape still names the expert and row counts."""
    E, N = b.shape[0], b.shape[1]
    src = b.contiguous().view(torch.uint8).reshape(E, N, -1)
    out = torch.empty_like(src)
    _lib.check(_lib.load().bsf_tile_weights(_ptr(src), E, N, src.shape[2], _ptr(out), _stream(stream)),
               "tile_weights")
    return out


def route_capacity(T: int, kr: int, E: int, layout: int, align_or_max_m: int) -> int:
    """Worst-case packed row count (no device-to-host sync needed)."""
    if layout == MASKED:
        return E * align_or_max_m
    return T * kr + E * (align_or_max_m - 1)


class RouteBuffers:
    """Preallocated outputs of ``route`` / ``dispatch`` (reused across steps).  ``fmt`` picks the
    packed operand: "fp8" (a_packed [m_cap, K], sfa_packed [ceil(K/512), ld]) or "nvfp4"
    (a_packed [m_cap, K/2], sfa_packed [K/64, ld])."""

    def __init__(self, T, kr, E, layout, align_or_max_m, K=0, device="cuda", scatter=True, fmt="fp8"):
        self.T, self.kr, self.E, self.layout, self.align_or_max_m, self.K = T, kr, E, layout, align_or_max_m, K
        self.m_cap = route_capacity(T, kr, E, layout, align_or_max_m)
        i32 = dict(dtype=torch.int32, device=device)
        self.counts = torch.empty(E, **i32)
        self.seg_start = torch.empty(E + 1, **i32)
        self.output_index = torch.empty((T, kr), **i32)
        self.token_of_row = torch.empty(max(self.m_cap, 1), **i32)
        self.m_indices = torch.empty(max(self.m_cap, 1), **i32)
        ws = _lib.load().bsf_route_workspace_bytes(T, kr, E)
        self.workspace = torch.empty(max(ws, 16), dtype=torch.uint8, device=device)
        self.fmt = fmt
        if scatter and K and fmt == "fp8_f32sf":
            self.a_packed = torch.empty((max(self.m_cap, 1), K), dtype=torch.uint8, device=device)
            self.sfa_packed = torch.empty((K // 128, sf_ld(self.m_cap)), dtype=torch.float32, device=device)
        elif scatter and K and fmt == "bf16":
            self.a_packed = torch.empty((max(self.m_cap, 1), K), dtype=torch.bfloat16, device=device)
            self.sfa_packed = None
        elif scatter and K and fmt == "nvfp4":
            self.a_packed = torch.empty((max(self.m_cap, 1), K // 2), dtype=torch.uint8, device=device)
            self.sfa_packed = torch.empty((K // 64, sf_ld(self.m_cap)), dtype=torch.int32, device=device)
        elif scatter and K:
            self.a_packed = torch.empty((max(self.m_cap, 1), K), dtype=torch.uint8, device=device)
            self.sfa_packed = torch.empty((sf_words(K), sf_ld(self.m_cap)), dtype=torch.int32, device=device)
        else:
            self.a_packed = self.sfa_packed = None


def route(topk_ids, E, layout, align_or_max_m, q=None, sf=None, bufs=None, stream=None, fmt="fp8"):
    """Routing + optional scatter of quantised rows (``fmt`` "fp8" or "nvfp4") or of bf16 rows
    (``fmt`` "bf16", ``q`` the bf16 activations, no ``sf``); returns a RouteBuffers."""
    T, kr = topk_ids.shape
    K = (q.shape[1] * (2 if fmt == "nvfp4" else 1)) if q is not None else 0
    if bufs is None:
        bufs = RouteBuffers(T, kr, E, layout, align_or_max_m, K=K, device=topk_ids.device, scatter=q is not None,
                            fmt=fmt)
    lib = _lib.load()
    if fmt == "bf16":
        _lib.check(lib.bsf_route_bf16(
            _ptr(topk_ids.contiguous()), T, kr, E, layout, align_or_max_m,
            _ptr(bufs.counts), _ptr(bufs.seg_start), _ptr(bufs.output_index), _ptr(bufs.token_of_row),
            _ptr(bufs.m_indices), bufs.m_cap, _ptr(q.contiguous() if q is not None else None), K,
            _ptr(bufs.a_packed) if q is not None else None, _ptr(bufs.workspace), bufs.workspace.numel(),
            _stream(stream)), "route_bf16")
        return bufs
    fn = {"nvfp4": lib.bsf_route_nvfp4, "fp8_f32sf": lib.bsf_route_f32sf}.get(fmt, lib.bsf_route)
    _lib.check(fn(
        _ptr(topk_ids.contiguous()), T, kr, E, layout, align_or_max_m,
        _ptr(bufs.counts), _ptr(bufs.seg_start), _ptr(bufs.output_index), _ptr(bufs.token_of_row),
        _ptr(bufs.m_indices), bufs.m_cap,
        _ptr(q), _ptr(sf), sf.shape[1] if sf is not None else 0, K,
        _ptr(bufs.a_packed) if q is not None else None, _ptr(bufs.sfa_packed) if q is not None else None,
        bufs.sfa_packed.shape[1] if (q is not None and bufs.sfa_packed is not None) else 0,
        _ptr(bufs.workspace), bufs.workspace.numel(), _stream(stream)), "route")
    return bufs


DISPATCH_MAX_ASSIGNMENTS = 16384
DISPATCH_MAX_EXPERTS = 256


def dispatch_supported(T, kr, E):
    return T * kr <= DISPATCH_MAX_ASSIGNMENTS and E <= DISPATCH_MAX_EXPERTS


def dispatch(x, topk_ids, E, layout, align_or_max_m, bufs=None, stream=None):
    """Quantise + route + scatter in one launch (small batches); returns a RouteBuffers."""
    T, K = x.shape
    kr = topk_ids.shape[1]
    if bufs is None:
        bufs = RouteBuffers(T, kr, E, layout, align_or_max_m, K=K, device=x.device)
    _lib.check(_lib.load().bsf_dispatch(
        _ptr(x.contiguous()), T, K, _ptr(topk_ids.contiguous()), kr, E, layout, align_or_max_m,
        _ptr(bufs.counts), _ptr(bufs.seg_start), _ptr(bufs.output_index), _ptr(bufs.token_of_row),
        _ptr(bufs.m_indices), bufs.m_cap, _ptr(bufs.a_packed), _ptr(bufs.sfa_packed), bufs.sfa_packed.shape[1],
        _stream(stream)), "dispatch")
    return bufs


def route_quantise_supported(kr):
    return kr <= 32


def route_quantise(x, topk_ids, E, layout, align_or_max_m, bufs=None, stream=None):
    """Quantise + route + scatter for batches of any size (routing kernels, then each token's row
    quantised once and written to its k_r packed rows); returns a RouteBuffers."""
    T, K = x.shape
    kr = topk_ids.shape[1]
    if bufs is None:
        bufs = RouteBuffers(T, kr, E, layout, align_or_max_m, K=K, device=x.device)
    _lib.check(_lib.load().bsf_route_quantise(
        _ptr(x.contiguous()), T, K, _ptr(topk_ids.contiguous()), kr, E, layout, align_or_max_m,
        _ptr(bufs.counts), _ptr(bufs.seg_start), _ptr(bufs.output_index), _ptr(bufs.token_of_row),
        _ptr(bufs.m_indices), bufs.m_cap, _ptr(bufs.a_packed), _ptr(bufs.sfa_packed), bufs.sfa_packed.shape[1],
        _ptr(bufs.workspace), bufs.workspace.numel(), _stream(stream)), "route_quantise")
    return bufs


def grouped_gemm_contig(a, sfa, b, sfb, seg_start, counts, d=None, flags=0, stream=None):
    """a uint8 [m_cap, K], b uint8 [E, N, K] -> d bf16 [m_cap, N] (segment rows written)."""
    m_cap, K = a.shape
    E, N, _ = b.shape
    if d is None:
        d = torch.empty((m_cap, N), dtype=torch.bfloat16, device=a.device)
    _lib.check(_lib.load().bsf_grouped_gemm_contig(
        _ptr(a), _ptr(sfa), sfa.shape[1], m_cap, _wptr(b, flags), _wptr(sfb, flags), _ptr(d), _ptr(seg_start), _ptr(counts),
        E, N, K, flags, _stream(stream)), "grouped_gemm_contig")
    return d


def grouped_gemm_masked(a, sfa, b, sfb, masked_m, max_m, d=None, expected_m=0, flags=0, stream=None):
    """a uint8 [E*max_m, K] (or [E, max_m, K]), b uint8 [E, N, K] -> d bf16 [E*max_m, N]."""
    K = a.shape[-1]
    E, N, _ = b.shape
    if d is None:
        d = torch.empty((E * max_m, N), dtype=torch.bfloat16, device=a.device)
    _lib.check(_lib.load().bsf_grouped_gemm_masked(
        _ptr(a), _ptr(sfa), sfa.shape[1], _wptr(b, flags), _wptr(sfb, flags), _ptr(d), _ptr(masked_m), E, max_m, N, K,
        expected_m, flags, _stream(stream)), "grouped_gemm_masked")
    return d


def combine(y, output_index, topk_weights, z=None, stream=None):
    """y bf16 [rows, N] -> z bf16 [T, N]."""
    rows, N = y.shape
    T, kr = output_index.shape
    if z is None:
        z = torch.empty((T, N), dtype=torch.bfloat16, device=y.device)
    _lib.check(_lib.load().bsf_combine(
        _ptr(y), rows, _ptr(output_index.contiguous()), _ptr(topk_weights.contiguous()), T, kr, N, _ptr(z),
        _stream(stream)), "combine")
    return z


def checksum_u64(t, host_mapped=False, out=None, stream=None):
    """XOR of the 64-bit words of a tensor's bytes (device tensor, or pinned host tensor if host_mapped)."""
    nbytes = t.numel() * t.element_size()
    if out is None:
        out = torch.empty(1, dtype=torch.int64, device="cuda")
    _lib.check(_lib.load().bsf_checksum_u64(_wptr(t, B_HOST_MAPPED if host_mapped else 0), nbytes,
                                            B_HOST_MAPPED if host_mapped else 0, _ptr(out),
                                            _stream(stream)), "checksum_u64")
    return out


# ----------------------------------------------------------------------------- NVFP4
def nvfp4_tensor_exponent(x, groups=1, out=None, stream=None):
    """Least j per group with max|x| <= 6 * 448 * 2**j; x bf16 split into ``groups`` equal groups."""
    x = x.contiguous()
    if out is None:
        out = torch.empty(groups, dtype=torch.int32, device=x.device)
    _lib.check(_lib.load().bsf_nvfp4_tensor_exponent(_ptr(x), groups, x.numel() // groups, _ptr(out),
                                                     _stream(stream)), "nvfp4_tensor_exponent")
    return out


def quantise_act_nvfp4(x, a_exp=0, q=None, sf=None, stream=None):
    """x bf16 [T, K] -> (q uint8 [T, K/2], sf int32 [K/64, sf_ld(T)])."""
    T, K = x.shape
    if q is None:
        q = torch.empty((T, K // 2), dtype=torch.uint8, device=x.device)
    if sf is None:
        sf = torch.empty((K // 64, sf_ld(T)), dtype=torch.int32, device=x.device)
    _lib.check(_lib.load().bsf_quantise_act_nvfp4(_ptr(x.contiguous()), T, K, int(a_exp), _ptr(q), _ptr(sf),
                                                  sf.shape[1], _stream(stream)), "quantise_act_nvfp4")
    return q, sf


def quantise_weight_nvfp4(w, b_exp=None, stream=None):
    """w bf16 [E, N, K] -> (q uint8 [E, N, K/2], sfb int32 [E, K/64, N], b_exp int32 [E]).
    Without ``b_exp`` each expert takes its least tensor exponent (``nvfp4_tensor_exponent``)."""
    E, N, K = w.shape
    w = w.contiguous()
    if b_exp is None:
        b_exp = nvfp4_tensor_exponent(w, groups=E, stream=stream)
    q = torch.empty((E, N, K // 2), dtype=torch.uint8, device=w.device)
    sfb = torch.empty((E, K // 64, N), dtype=torch.int32, device=w.device)
    _lib.check(_lib.load().bsf_quantise_weight_nvfp4(_ptr(w), E, N, K, _ptr(b_exp), _ptr(q), _ptr(sfb),
                                                     _stream(stream)), "quantise_weight_nvfp4")
    return q, sfb, b_exp


def dispatch_nvfp4(x, topk_ids, E, layout, align_or_max_m, a_exp=0, bufs=None, stream=None):
    """NVFP4 quantise + route + scatter in one launch (small batches); returns a RouteBuffers."""
    T, K = x.shape
    kr = topk_ids.shape[1]
    if bufs is None:
        bufs = RouteBuffers(T, kr, E, layout, align_or_max_m, K=K, device=x.device, fmt="nvfp4")
    _lib.check(_lib.load().bsf_dispatch_nvfp4(
        _ptr(x.contiguous()), T, K, int(a_exp), _ptr(topk_ids.contiguous()), kr, E, layout, align_or_max_m,
        _ptr(bufs.counts), _ptr(bufs.seg_start), _ptr(bufs.output_index), _ptr(bufs.token_of_row),
        _ptr(bufs.m_indices), bufs.m_cap, _ptr(bufs.a_packed), _ptr(bufs.sfa_packed), bufs.sfa_packed.shape[1],
        _stream(stream)), "dispatch_nvfp4")
    return bufs


def grouped_gemm_nvfp4_contig(a, sfa, a_exp, b, sfb, b_exp, seg_start, counts, d=None, flags=0, stream=None):
    """a uint8 [m_cap, K/2], b uint8 [E, N, K/2] -> d bf16 [m_cap, N] (segment rows written)."""
    m_cap, K2 = a.shape
    E, N, _ = b.shape
    if d is None:
        d = torch.empty((m_cap, N), dtype=torch.bfloat16, device=a.device)
    _lib.check(_lib.load().bsf_grouped_gemm_nvfp4_contig(
        _ptr(a), _ptr(sfa), sfa.shape[1], m_cap, int(a_exp), _wptr(b, flags), _wptr(sfb, flags), _ptr(b_exp), _ptr(d),
        _ptr(seg_start), _ptr(counts), E, N, 2 * K2, flags, _stream(stream)), "grouped_gemm_nvfp4_contig")
    return d


def grouped_gemm_nvfp4_masked(a, sfa, a_exp, b, sfb, b_exp, masked_m, max_m, d=None, expected_m=0, flags=0,
                              stream=None):
    """a uint8 [E*max_m, K/2], b uint8 [E, N, K/2] -> d bf16 [E*max_m, N]."""
    K2 = a.shape[-1]
    E, N, _ = b.shape
    if d is None:
        d = torch.empty((E * max_m, N), dtype=torch.bfloat16, device=a.device)
    _lib.check(_lib.load().bsf_grouped_gemm_nvfp4_masked(
        _ptr(a), _ptr(sfa), sfa.shape[1], int(a_exp), _wptr(b, flags), _wptr(sfb, flags), _ptr(b_exp), _ptr(d), _ptr(masked_m),
        E, max_m, N, 2 * K2, expected_m, flags, _stream(stream)), "grouped_gemm_nvfp4_masked")
    return d


# ----------------------------------------------------------------------------- BF16
def grouped_gemm_bf16_contig(a, b, seg_start, counts, d=None, flags=0, stream=None):
    """a bf16 [m_cap, K], b bf16 [E, N, K] -> d bf16 [m_cap, N] (segment rows written)."""
    m_cap, K = a.shape
    E, N, _ = b.shape
    if d is None:
        d = torch.empty((m_cap, N), dtype=torch.bfloat16, device=a.device)
    _lib.check(_lib.load().bsf_grouped_gemm_bf16_contig(
        _ptr(a), m_cap, _wptr(b, flags), _ptr(d), _ptr(seg_start), _ptr(counts), E, N, K, flags, _stream(stream)),
        "grouped_gemm_bf16_contig")
    return d


def grouped_gemm_bf16_masked(a, b, masked_m, max_m, d=None, expected_m=0, flags=0, stream=None):
    """a bf16 [E*max_m, K], b bf16 [E, N, K] -> d bf16 [E*max_m, N]."""
    K = a.shape[-1]
    E, N, _ = b.shape
    if d is None:
        d = torch.empty((E * max_m, N), dtype=torch.bfloat16, device=a.device)
    _lib.check(_lib.load().bsf_grouped_gemm_bf16_masked(
        _ptr(a), _wptr(b, flags), _ptr(d), _ptr(masked_m), E, max_m, N, K, expected_m, flags, _stream(stream)),
        "grouped_gemm_bf16_masked")
    return d


# ----------------------------------------------------------------------------- FP8 with float32 scales
def quantise_act_f32sf(x, q=None, sf=None, stream=None):
    """x bf16 [T, K] -> (q uint8 [T, K], sf float32 [K/128, sf_ld(T)])."""
    T, K = x.shape
    if q is None:
        q = torch.empty((T, K), dtype=torch.uint8, device=x.device)
    if sf is None:
        sf = torch.empty((K // 128, sf_ld(T)), dtype=torch.float32, device=x.device)
    _lib.check(_lib.load().bsf_quantise_act_f32sf(_ptr(x.contiguous()), T, K, _ptr(q), _ptr(sf), sf.shape[1],
                                                  _stream(stream)), "quantise_act_f32sf")
    return q, sf


def quantise_weight_f32sf(w, stream=None):
    """w bf16 [E, N, K] -> (q uint8 [E, N, K], sf float32 [E, N/128, K/128])."""
    E, N, K = w.shape
    q = torch.empty((E, N, K), dtype=torch.uint8, device=w.device)
    sf = torch.empty((E, N // 128, K // 128), dtype=torch.float32, device=w.device)
    _lib.check(_lib.load().bsf_quantise_weight_f32sf(_ptr(w.contiguous()), E, N, K, _ptr(q), _ptr(sf),
                                                     _stream(stream)), "quantise_weight_f32sf")
    return q, sf


def grouped_gemm_f32sf_contig(a, sfa, b, sfb, seg_start, counts, d=None, flags=0, stream=None):
    """a uint8 [m_cap, K], sfa float32 [K/128, ld], b uint8 [E, N, K], sfb float32 [E, N/128, K/128]."""
    m_cap, K = a.shape
    E, N, _ = b.shape
    if d is None:
        d = torch.empty((m_cap, N), dtype=torch.bfloat16, device=a.device)
    _lib.check(_lib.load().bsf_grouped_gemm_f32sf_contig(
        _ptr(a), _ptr(sfa), sfa.shape[1], m_cap, _wptr(b, flags), _wptr(sfb, flags), _ptr(d), _ptr(seg_start), _ptr(counts),
        E, N, K, flags, _stream(stream)), "grouped_gemm_f32sf_contig")
    return d


def grouped_gemm_f32sf_masked(a, sfa, b, sfb, masked_m, max_m, d=None, expected_m=0, flags=0, stream=None):
    """a uint8 [E*max_m, K], sfa float32 [K/128, ld] -> d bf16 [E*max_m, N]."""
    K = a.shape[-1]
    E, N, _ = b.shape
    if d is None:
        d = torch.empty((E * max_m, N), dtype=torch.bfloat16, device=a.device)
    _lib.check(_lib.load().bsf_grouped_gemm_f32sf_masked(
        _ptr(a), _ptr(sfa), sfa.shape[1], _wptr(b, flags), _wptr(sfb, flags), _ptr(d), _ptr(masked_m), E, max_m, N, K, expected_m,
        flags, _stream(stream)), "grouped_gemm_f32sf_masked")
    return d


# ----------------------------------------------------------------------------- around the expert path
GATE_SIGMOID = 0x1
GATE_GROUP_TOP2 = 0x2
GATE_RENORMALISE = 0x4
_TYPES = {torch.float32: 0, torch.bfloat16: 1}       # BSF_TYPE_F32, BSF_TYPE_BF16
_SCORES = {"softmax": 0, "sigmoid": GATE_SIGMOID}
_GROUP_SCORES = {"max": 0, "top2": GATE_GROUP_TOP2}


# The checks of these operators are written out in the calls rather than shared: on a call of a few
# microseconds every attribute of a tensor that is read, and every Python call, is a tenth of one.
def _refuse(t, dtype, shape, what):
    """Why tensor ``t`` is not a contiguous CUDA tensor of this type and shape."""
    if t.dtype != dtype:
        raise ValueError(f"{what}: expected {dtype}, got {t.dtype}")
    if shape is not None and (t.shape != shape or not t.is_contiguous()):
        raise ValueError(f"{what}: expected a contiguous tensor of shape {tuple(shape)}, got {tuple(t.shape)}")
    raise ValueError(f"{what}: expected a CUDA tensor, got one on {t.device}")


def _row_stride(t, rows, cols, what):
    """Row stride of a 2-D tensor whose rows are contiguous.  That of a single row is never used: whatever the
    view says (logits[:, -1] of one sequence strides over all of it), the next multiple of 8 is in every range."""
    ld, step = t.stride()
    if step != 1 and cols > 1:
        raise ValueError(f"{what}: expected a 2-D tensor with contiguous rows")
    return ld if rows > 1 else (cols + 7) // 8 * 8


def _two_dims(t, what):
    if t.dim() != 2:
        raise ValueError(f"{what}: expected a 2-D tensor with contiguous rows, got {t.dim()} dimensions")
    return t.shape


def _used_on(stream, *tensors):
    """The allocator keeps the memory of these tensors until the work queued on ``stream`` is done, also if the
    caller drops them at once."""
    for t in tensors:
        if t is not None:
            t.record_stream(stream)


def _empty(shape, dtype, like, stream):
    """An output that ``stream`` (None: the current one) writes.  Memory that the current stream freed may still
    be in use there, so another stream takes its own; the current stream is where the caller will use it."""
    if stream is None or not like.is_cuda:
        return torch.empty(shape, dtype=dtype, device=like.device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=like.device)
    t.record_stream(torch.cuda.current_stream(like.device))
    return t


_F32, _BF16, _I32, _U8 = torch.float32, torch.bfloat16, torch.int32, torch.uint8
# handle of a device's current stream, without making a stream object (2.8 us of a call)
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda device: torch.cuda.current_stream(device).cuda_stream)


# index of the device that the library launches on and whose SM count and error word it uses
_current_device = torch._C._cuda_getDevice


def _refuse_devices(names, operands, stream):
    """Why these operands (None: not given) are not all on the current CUDA device."""
    for name, t in zip(names.split(), operands):
        if t is not None and not t.is_cuda:
            raise ValueError(f"{name}: expected a CUDA tensor, got one on {t.device}")
    on = [f"{name} on {t.device}" for name, t in zip(names.split(), operands) if t is not None]
    if stream is not None:
        on.append(f"stream on cuda:{stream.device_index}")
    raise ValueError(f"expected every operand on the current device cuda:{_current_device()}: {', '.join(on)}")


def gate(logits, kr, score="softmax", bias=None, groups=1, kept_groups=None, group_score="max", renormalise=True,
         scale=1.0, topk_ids=None, topk_weights=None, stream=None):
    """Router logits [T, E] (float32 or bf16, any row stride) -> (topk_ids int32 [T, kr], topk_weights
    float32 [T, kr]) for ``route`` / ``dispatch`` / ``combine``.  ``score`` "softmax" or "sigmoid"; with
    ``bias`` float32 [E] the choice goes by score + bias; of ``groups`` groups of experts only the
    ``kept_groups`` best take part (``group_score`` "max" or "top2"); ids of -1 where too few experts can
    be chosen (a logit of -inf or NaN masks its expert)."""
    kind = _TYPES.get(logits.dtype)
    if kind is None:
        raise ValueError(f"logits: expected float32 or bfloat16, got {logits.dtype}")
    if score not in _SCORES or group_score not in _GROUP_SCORES:
        raise ValueError(f"score {score!r} / group_score {group_score!r}: expected softmax or sigmoid / max or top2")
    T, E = _two_dims(logits, "logits")
    ld = _row_stride(logits, T, E, "logits")
    out = (T, kr)
    if topk_ids is None:
        topk_ids = _empty(out, _I32, logits, stream)
    elif topk_ids.dtype != _I32 or topk_ids.shape != out or not topk_ids.is_contiguous():
        _refuse(topk_ids, _I32, out, "topk_ids")
    if topk_weights is None:
        topk_weights = _empty(out, _F32, logits, stream)
    elif topk_weights.dtype != _F32 or topk_weights.shape != out or not topk_weights.is_contiguous():
        _refuse(topk_weights, _F32, out, "topk_weights")
    if bias is not None:
        if bias.dtype != _F32 or bias.shape != (E,) or not bias.is_contiguous() or not bias.is_cuda:
            _refuse(bias, _F32, (E,), "bias")
    device = logits.get_device()               # (-1 of a host tensor)
    if (device < 0 or topk_ids.get_device() != device or topk_weights.get_device() != device
            or (bias is not None and bias.get_device() != device) or device != _current_device()
            or (stream is not None and stream.device_index != device)):
        _refuse_devices("logits topk_ids topk_weights bias", (logits, topk_ids, topk_weights, bias), stream)
    if stream is not None:
        _used_on(stream, logits, topk_ids, topk_weights, bias)
    status = _lib.load().bsf_gate(
        logits.data_ptr(), kind, T, E, ld, None if bias is None else bias.data_ptr(), groups, groups if kept_groups is None else kept_groups, kr,
        _SCORES[score] | _GROUP_SCORES[group_score] | (GATE_RENORMALISE if renormalise else 0), scale,
        topk_ids.data_ptr(), topk_weights.data_ptr(),
        _current_stream(device) if stream is None else stream.cuda_stream)
    if status:
        _lib.check(status, "gate")
    return topk_ids, topk_weights


def swiglu_quantise(y, rows=None, q=None, sf=None, stream=None):
    """y bf16 [T, 2 K] (gate columns, then up columns; any row stride that is a multiple of 8) ->
    (q uint8 [T, Kp], sf int32 [ceil(Kp/512), >= T]) of silu(gate) * up, Kp = K rounded up to 128.
    ``rows`` as in ``quantise_act``: only the routed rows of a packed operand."""
    T, K = _two_dims(y, "y")
    ld = _row_stride(y, T, K, "y")
    if K % 2:
        raise ValueError(f"y: expected an even number of columns, got {K}")
    if y.dtype != _BF16:
        _refuse(y, _BF16, None, "y")
    K //= 2
    Kp = (K + 127) // 128 * 128
    words = (Kp + 511) // 512
    if q is None:
        q = _empty((T, Kp), _U8, y, stream)
    elif q.dtype != _U8 or q.shape != (T, Kp) or not q.is_contiguous():
        _refuse(q, _U8, (T, Kp), "q")
    if sf is None:
        sf = _empty((words, sf_ld(T)), _I32, y, stream)
    ld_sf = sf.shape[-1]
    if sf.dtype != _I32 or sf.shape != (words, ld_sf) or not sf.is_contiguous():
        _refuse(sf, _I32, (words, ld_sf), "sf")
    token_of_row = rows_used = None
    if rows is not None:
        token_of_row, rows_used = rows
        if (token_of_row.dtype != _I32 or rows_used.dtype != _I32 or token_of_row.numel() < T or rows_used.numel() < 1
                or not token_of_row.is_cuda or not rows_used.is_cuda or not token_of_row.is_contiguous()):
            raise ValueError("rows: expected CUDA int32 tensors, token_of_row of at least T entries and rows_used of one")
    device = y.get_device()
    if (device < 0 or q.get_device() != device or sf.get_device() != device
            or (rows is not None and (token_of_row.get_device() != device or rows_used.get_device() != device))
            or device != _current_device() or (stream is not None and stream.device_index != device)):
        _refuse_devices("y q sf token_of_row rows_used", (y, q, sf, token_of_row, rows_used), stream)
    if stream is not None:
        _used_on(stream, y, q, sf, token_of_row, rows_used)
    status = _lib.load().bsf_swiglu_quantise(
        y.data_ptr(), T, K, ld, None if rows is None else token_of_row.data_ptr(),
        None if rows is None else rows_used.data_ptr(), q.data_ptr(), sf.data_ptr(), ld_sf,
        _current_stream(device) if stream is None else stream.cuda_stream)
    if status:
        _lib.check(status, "swiglu_quantise")
    return q, sf


def prepare_dense_weight(w):
    """w bf16 [N, K] -> (b uint8 [Np, Kp] tiled, sfb int32 [ceil(Kp/512), Np]) for ``dense_gemm`` with
    ``B_TILED``, on the current stream; N and K are rounded up to 128 with zero weights."""
    N, K = _two_dims(w, "w")
    if w.dtype != _BF16 or not w.is_cuda:
        _refuse(w, _BF16, None, "w")
    w = torch.nn.functional.pad(w, (0, -K % 128, 0, -N % 128))
    q, sf128 = quantise_weight(w.unsqueeze(0))
    sfb = prepare_weight_sf(sf128, w.shape[1])
    return tile_weights(q)[0], sfb[0]


def dense_gemm(a, sfa, b, sfb, N=None, addend=None, d=None, flags=B_TILED, stream=None):
    """a uint8 [M, K] with scales sfa, b uint8 [Np, K] with scales sfb (``prepare_dense_weight``) ->
    d bf16 [M, N], N <= Np < N + 128 (default Np); ``addend`` bf16 [M, N] is added before the rounding."""
    M, K = _two_dims(a, "a")
    Np = b.shape[0]
    N = Np if N is None else N
    if (N + 127) // 128 * 128 != Np:
        raise ValueError(f"b: expected {(N + 127) // 128 * 128} rows for N = {N}, got {Np}")
    words, ld_sf = (K + 511) // 512, sfa.shape[-1]
    if a.dtype != _U8 or not a.is_contiguous():
        _refuse(a, _U8, (M, K), "a")
    if b.dtype != _U8 or b.shape != (Np, K) or not b.is_contiguous():
        _refuse(b, _U8, (Np, K), "b")
    if sfa.dtype != _I32 or sfa.shape != (words, ld_sf) or not sfa.is_contiguous():
        _refuse(sfa, _I32, (words, ld_sf), "sfa")
    if sfb.dtype != _I32 or sfb.shape != (words, Np) or not sfb.is_contiguous():
        _refuse(sfb, _I32, (words, Np), "sfb")
    out = (M, N)
    if d is None:
        d = _empty(out, _BF16, a, stream)
    elif d.dtype != _BF16 or d.shape != out:
        _refuse(d, _BF16, out, "d")
    ldd = _row_stride(d, M, N, "d")
    ldc = 0
    if addend is not None:
        if addend.dtype != _BF16 or addend.shape != out or not addend.is_cuda:
            _refuse(addend, _BF16, out, "addend")
        ldc = _row_stride(addend, M, N, "addend")
    device = a.get_device()
    if (device < 0 or sfa.get_device() != device or b.get_device() != device or sfb.get_device() != device
            or d.get_device() != device or (addend is not None and addend.get_device() != device)
            or device != _current_device() or (stream is not None and stream.device_index != device)):
        _refuse_devices("a sfa b sfb d addend", (a, sfa, b, sfb, d, addend), stream)
    if stream is not None:
        _used_on(stream, a, sfa, b, sfb, d, addend)
    status = _lib.load().bsf_dense_gemm(
        a.data_ptr(), sfa.data_ptr(), ld_sf, M, b.data_ptr(), sfb.data_ptr(), N, K,
        None if addend is None else addend.data_ptr(), ldc, d.data_ptr(), ldd, flags,
        _current_stream(device) if stream is None else stream.cuda_stream)
    if status:
        _lib.check(status, "dense_gemm")
    return d
