"""Cases for the operators around the expert path of an MoE block: router choice (``gate``), SwiGLU into the
quantised operand of the next product (``swiglu``) and the dense FP8 product of an always-active expert
(``dense``).

``run`` computes them with elementary torch operations in float32 (``own`` false) or calls the package's
operators (``own`` true); ``exact`` computes them in 64 bits from their definitions.
"""

import math

import numpy as np
import torch

own = False

DEV = "cuda"
FLT_MAX = torch.finfo(torch.float32).max


# ----------------------------------------------------------------------------- cases
def listed():
    return [
        # router of one decoded token: 256 experts, balance bias, 4 of 16 groups kept
        dict(name="gate_one_token", op="gate", T=1, E=256, kr=8, dtype="f32", score="sigmoid", bias=True, groups=16,
             kept=4, group_score="top2", renormalise=True, scale=2.5, masked=0.0),
        # a decode batch padded to a fixed graph size: the padding rows' logits are all -inf
        dict(name="gate_decode", op="gate", T=128, E=128, kr=8, dtype="bf16", score="softmax", bias=False, groups=1,
             kept=1, group_score="max", renormalise=True, scale=1.0, masked=0.05),
        # one large prefill batch through a balanced router
        dict(name="gate_large", op="gate", T=8192, E=256, kr=8, dtype="f32", score="sigmoid", bias=True, groups=16,
             kept=4, group_score="top2", renormalise=True, scale=2.5, masked=0.0),
        # all tokens of a long packed batch, odd counts, group-limited softmax router without renormalisation
        dict(name="gate_long", op="gate", T=65533, E=192, kr=6, dtype="f32", score="softmax", bias=False, groups=8,
             kept=3, group_score="max", renormalise=False, scale=16.0, masked=0.0),
        # always-active expert of a few decoded tokens, width not a multiple of the scale block
        dict(name="swiglu_few_tokens", op="swiglu", T=5, K=1416, kr=1, E=0, align=1),
        # routed rows of a decode batch in masked slots of 64 rows (128 experts, top 8): most rows are padding
        dict(name="swiglu_decode_slots", op="swiglu", T=128, K=1536, kr=8, E=128, align=0),
        # routed rows of a large batch in segments padded to 128 rows (256 experts, top 8)
        dict(name="swiglu_large", op="swiglu", T=8192, K=2048, kr=8, E=256, align=128),
        # gate-up product of an always-active expert for one token: the weights stream once
        dict(name="dense_one_token", op="dense", M=1, N=4096, K=7168, addend=False),
        # down product for a small ragged batch, added to the routed experts' sum
        dict(name="dense_small_batch", op="dense", M=37, N=7168, K=2048, addend=True),
        # decode batch, the decode workload's shape as one dense layer
        dict(name="dense_decode", op="dense", M=128, N=3072, K=4096, addend=False),
        # a prefill chunk between two tile sizes, output width not a multiple of 128
        dict(name="dense_chunk", op="dense", M=777, N=2112, K=7168, addend=False),
        # gate-up product of an always-active expert over a large prefill batch
        dict(name="dense_large", op="dense", M=8192, N=4096, K=7168, addend=False),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["gate", "swiglu", "dense"])
    if op == "gate":
        groups = rng.choice([1, 1, 2, 4, 8, 16])
        per = rng.choice([4, 5, 8, 12, 16, 20, 32]) if groups > 1 else rng.randint(8, 500)
        per = min(per, 512 // groups)
        kept = rng.randint(max(1, groups // 4), groups)
        E = groups * per
        T = min(_log_int(rng, 1, 60000), 16000000 // E)
        return dict(op="gate", T=T, E=E, kr=min(rng.randint(1, 10), kept * per), dtype=rng.choice(["f32", "bf16"]),
                    score=rng.choice(["softmax", "sigmoid"]), bias=rng.random() < 0.5, groups=groups, kept=kept,
                    group_score=rng.choice(["max", "top2"]), renormalise=rng.random() < 0.6,
                    scale=rng.choice([1.0, 2.5]), masked=rng.choice([0.0, 0.03]))
    if op == "swiglu":
        K = 8 * _log_int(rng, 16, 512)
        kind = rng.choice(["plain", "masked", "segments"])
        if kind == "plain":
            return dict(op="swiglu", T=min(_log_int(rng, 1, 60000), 120000000 // K), K=K, kr=1, E=0, align=1)
        E = rng.choice([8, 32, 128])
        kr = rng.choice([2, 4, 8])
        T = _log_int(rng, 1, 128) if kind == "masked" else min(_log_int(rng, 16, 8192), 100000000 // (K * kr))
        return dict(op="swiglu", T=T, K=K, kr=kr, E=E, align=0 if kind == "masked" else 128)
    while True:
        M, N, K = _log_int(rng, 1, 8192), _log_int(rng, 64, 8192), 128 * _log_int(rng, 2, 56)
        if M * N * K <= 8192 * 4096 * 7168:
            return dict(op="dense", M=M, N=N, K=K, addend=rng.random() < 0.4)


def _padded(n):
    return (n + 127) // 128 * 128


def _segments(case):
    """Packed rows of a routed swiglu case: masked slots of 64 rows, or aligned segments."""
    if case["align"] == 0:
        return case["E"] * 64
    return case["T"] * case["kr"] + case["E"] * (case["align"] - 1)


def work(case):
    if case["op"] == "gate":
        size = 4 if case["dtype"] == "f32" else 2
        T, E, kr = case["T"], case["E"], case["kr"]
        return {"bytes": T * E * size + T * kr * 8 + (4 * E if case["bias"] else 0), "flops": 6 * T * E}
    if case["op"] == "swiglu":
        K, rows = case["K"], case["T"] * case["kr"]
        rows = min(rows, case["E"] * 64) if case["E"] and case["align"] == 0 else rows
        words = (_padded(K) // 128 + 3) // 4
        marks = 4 * _segments(case) if case["E"] else 0
        return {"bytes": rows * (4 * K + _padded(K) + 4 * words) + marks, "flops": 8 * rows * K}
    M, N, K = case["M"], case["N"], case["K"]
    words = (K // 128 + 3) // 4
    return {"bytes": M * K + N * K + 4 * words * (M + N) + M * N * (4 if case["addend"] else 2),
            "flops": 2 * M * N * K}


# ----------------------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _close_calls(logits, bias, case):
    """Rows whose choice hangs on the last bits of a float32 score (keys or group scores nearer than 4e-6 at a
    place where their order matters).  Where the keys are the logits themselves no order is ever unclear."""
    T, E = logits.shape
    G, kr = case["groups"], case["kr"]
    by_logit = bias is None
    if by_logit and (G == 1 or case["group_score"] == "max"):
        return torch.zeros(T, dtype=torch.bool, device=DEV)
    l = logits.double()
    s = torch.sigmoid(l) if case["score"] == "sigmoid" else torch.softmax(l, 1)
    s = torch.nan_to_num(s, nan=0.0)
    key = s if bias is None else s + bias.double()
    bad = torch.zeros(T, dtype=torch.bool, device=DEV)
    allowed = torch.ones_like(key, dtype=torch.bool)
    if G > 1:
        per = key.view(T, G, E // G)
        gs = per.amax(2) if case["group_score"] == "max" else per.sort(dim=2, descending=True)[0][:, :, :2].sum(2)
        srt, order = gs.sort(dim=1, descending=True)
        if case["kept"] < G:
            bad |= srt[:, case["kept"] - 1] - srt[:, case["kept"]] < 4e-6
        keep = torch.zeros_like(gs, dtype=torch.bool).scatter_(1, order[:, :case["kept"]], True)
        allowed = keep.repeat_interleave(E // G, dim=1)
    if not by_logit:
        top = torch.where(allowed, key, -math.inf).sort(dim=1, descending=True)[0][:, :kr + 1]
        bad |= (top[:, :-1] - top[:, 1:] < 4e-6).any(1)
    return bad


def _prepare_gate(case, seed):
    g = _gen(seed)
    T, E = case["T"], case["E"]
    dtype = torch.float32 if case["dtype"] == "f32" else torch.bfloat16
    # a trained router's logits: unit noise on a per-expert popularity; the balance bias is a small correction
    popularity = 0.5 * torch.randn(E, device=DEV, generator=g)
    bias = 0.05 * torch.randn(E, device=DEV, generator=g) if case["bias"] else None
    logits = (popularity + torch.randn(T, E, device=DEV, generator=g)).to(dtype)
    for _ in range(12):
        bad = _close_calls(logits, bias, case).nonzero().flatten()
        if bad.numel() == 0:
            break
        logits[bad] = (popularity + torch.randn(bad.numel(), E, device=DEV, generator=g)).to(dtype)
    if case["masked"]:
        pad = torch.rand(T, device=DEV, generator=g) < case["masked"]
        pad[T - 1] = True                                  # at least one row offers no expert at all
        logits[pad] = -math.inf
    ids = torch.zeros(T, case["kr"], dtype=torch.int32, device=DEV)
    weights = torch.zeros(T, case["kr"], dtype=torch.float32, device=DEV)
    return dict(case=case, logits=logits, bias=bias, ids=ids, weights=weights)


def _prepare_swiglu(case, seed):
    g = _gen(seed)
    K, T, kr, E = case["K"], case["T"], case["kr"], case["E"]
    rows = None
    if E == 0:
        R = T
    else:
        R = _segments(case)
        # every token's kr distinct experts, by the largest of E random scores
        picks = torch.rand(T, E, device=DEV, generator=g).topk(kr, dim=1)[1]
        counts = torch.bincount(picks.flatten(), minlength=E)
        r = torch.arange(R, device=DEV)
        if case["align"] == 0:
            counts = counts.clamp(max=64)
            starts = torch.arange(E + 1, device=DEV) * 64
        else:
            length = (counts + case["align"] - 1) // case["align"] * case["align"]
            starts = torch.cat([torch.zeros(1, dtype=torch.long, device=DEV), length.cumsum(0)])
        e = (torch.searchsorted(starts, r, right=True) - 1).clamp(max=E - 1)
        routed = (r - starts[e] < counts[e]) & (r < starts[E])
        token = torch.where(routed, r % T, -1)
        token = torch.where(r < starts[E], token, 0)       # rows past the last segment are never looked at
        rows = (token.int().contiguous(), starts[E:].int().contiguous())
    y = torch.randn(R, 2 * K, device=DEV, generator=g)
    y[:, :K] *= 1.5
    y[torch.rand(R, device=DEV, generator=g) < 0.01] *= 20.0   # outlier tokens
    y = y.to(torch.bfloat16)
    if rows is not None:                                   # padding rows hold whatever the memory held
        y[~routed] = math.nan
    words = (_padded(K) // 128 + 3) // 4
    q = torch.zeros(R, _padded(K), dtype=torch.uint8, device=DEV)
    sf = torch.zeros(words, (R + 3) // 4 * 4, dtype=torch.int32, device=DEV)
    return dict(case=case, y=y, rows=rows, q=q, sf=sf)


def _quantise(x, block_rows):
    """(E4M3 codes, exponents) of x over block_rows x 128 blocks: the least e with amax <= 448 * 2**e."""
    R, K = x.shape
    x = x.float()
    amax = x.abs().view(R // block_rows, block_rows, K // 128, 128).amax((1, 3))
    m, ex = torch.frexp(amax)
    e = torch.where(amax > 0, ex - 9 + (m > 0.875).int(), torch.zeros_like(ex)).clamp(-126, 127)
    scale = torch.ldexp(torch.ones_like(amax), -e)
    full = scale.repeat_interleave(block_rows, 0).repeat_interleave(128, 1)
    return (x * full).to(torch.float8_e4m3fn).view(torch.uint8), e


def _pack(e_rows, ld):
    """Exponents [rows, K/128] -> packed words [ceil(K/512), ld], byte j of word i for K-block 4 i + j."""
    rows, nkb = e_rows.shape
    words = (nkb + 3) // 4
    b = torch.full((words * 4, ld), 127, dtype=torch.int64, device=DEV)
    b[:nkb, :rows] = e_rows.t().long() + 127
    b = b.view(words, 4, ld)
    w = b[:, 0] | b[:, 1] << 8 | b[:, 2] << 16 | b[:, 3] << 24
    return torch.where(w >= 1 << 31, w - (1 << 32), w).int()


def _prepare_dense(case, seed):
    g = _gen(seed)
    M, N, K = case["M"], case["N"], case["K"]
    x = torch.randn(M, K, device=DEV, generator=g)
    x[torch.rand(M, device=DEV, generator=g) < 0.01] *= 50.0   # outlier tokens
    a, ea = _quantise(x.to(torch.bfloat16), 1)
    Np = _padded(N)
    w = torch.zeros(Np, K, device=DEV)
    w[:N] = 0.02 * torch.randn(N, K, device=DEV, generator=g)
    b, eb = _quantise(w.to(torch.bfloat16), 128)
    # the weights as a program keeps them: 128 x 128 blocks contiguous, one packed scale word per row and 512 K
    tiled = b.view(Np // 128, 128, K // 128, 128).permute(0, 2, 1, 3).contiguous().view(Np, K)
    addend = torch.randn(M, N, device=DEV, generator=g).to(torch.bfloat16) if case["addend"] else None
    d = torch.zeros(M, N, dtype=torch.bfloat16, device=DEV)
    return dict(case=case, a=a, sfa=_pack(ea, (M + 3) // 4 * 4), b=tiled, sfb=_pack(eb.repeat_interleave(128, 0), Np),
                addend=addend, d=d)


def prepare(case, seed):
    return {"gate": _prepare_gate, "swiglu": _prepare_swiglu, "dense": _prepare_dense}[case["op"]](case, seed)


# ----------------------------------------------------------------------------- one pass
def _plain_gate(s):
    c = s["case"]
    T, E, G, kr = c["T"], c["E"], c["groups"], c["kr"]
    l = s["logits"].float()
    usable = l > -math.inf
    l = torch.where(usable, l, 0.0).clamp(max=FLT_MAX)
    if c["score"] == "sigmoid":
        score = torch.where(usable, 1.0 / (1.0 + torch.exp(-l)), 0.0)
    else:
        m = torch.where(usable, l, -FLT_MAX).amax(1, keepdim=True)
        ex = torch.where(usable, torch.exp(l - m), 0.0)
        score = ex / ex.sum(1, keepdim=True).clamp(min=1e-37)
    key = l if s["bias"] is None else score + s["bias"]
    key = torch.where(usable, key, -math.inf)
    if G > 1:
        per = key.view(T, G, E // G)
        if c["group_score"] == "max":
            gs = per.amax(2)
        else:
            own_key = score if s["bias"] is None else score + s["bias"]
            two = torch.where(usable, own_key, -math.inf).view(T, G, E // G).sort(dim=2, descending=True)[0][:, :, :2]
            gs = two[:, :, 0] + (torch.where(two[:, :, 1] > -math.inf, two[:, :, 1], 0.0) if E > G else 0.0)
        order = gs.sort(dim=1, descending=True, stable=True)[1]
        keep = torch.zeros_like(gs, dtype=torch.bool).scatter_(1, order[:, :c["kept"]], True)
        key = torch.where(keep.view(T, G, 1), per, -math.inf).view(T, E)
    best, ids = key.sort(dim=1, descending=True, stable=True)
    best, ids = best[:, :kr], ids[:, :kr]
    w = torch.where(best > -math.inf, score.gather(1, ids), 0.0)
    if c["renormalise"]:
        total = w.sum(1, keepdim=True)
        w = torch.where(total > 0, w / total, 0.0)
    return {"ids": torch.where(best > -math.inf, ids, -1).int(), "weights": w * c["scale"]}


def _plain_swiglu(s):
    K, R = s["case"]["K"], s["y"].shape[0]
    y = s["y"].float()
    g, u = y[:, :K], y[:, K:]
    h = g / (1.0 + torch.exp(-g)) * u
    if s["rows"] is not None:
        token, used = s["rows"]
        routed = (token >= 0) & (torch.arange(R, device=DEV) < used)
        h = torch.where(routed.view(R, 1), h, 0.0)
    h = torch.nn.functional.pad(h, (0, _padded(K) - K))
    q, e = _quantise(h, 1)
    sf = _pack(e, s["sf"].shape[1])[:, :R]
    if s["rows"] is not None:                              # rows without a token stay unwritten
        sf = torch.where(routed, sf, 0)
    return {"q": q.view(torch.float8_e4m3fn), "sf": sf}


def _unpack(sf, rows, nkb):
    w = sf.long()
    b = torch.stack([w & 255, (w >> 8) & 255, (w >> 16) & 255, (w >> 24) & 255], 1).view(-1, sf.shape[1])
    return b[:nkb, :rows].t() - 127


def _plain_dense(s):
    c = s["case"]
    M, N, K = c["M"], c["N"], c["K"]
    Np = _padded(N)
    one = torch.ones((), device=DEV)
    a = s["a"].view(torch.float8_e4m3fn).float()
    a = a * torch.ldexp(one, _unpack(s["sfa"], M, K // 128)).repeat_interleave(128, 1)
    b = s["b"].view(Np // 128, K // 128, 128, 128).permute(0, 2, 1, 3).reshape(Np, K)[:N]
    b = b.contiguous().view(torch.float8_e4m3fn).float()
    b = b * torch.ldexp(one, _unpack(s["sfb"], N, K // 128)).repeat_interleave(128, 1)
    d = a @ b.t()
    if s["addend"] is not None:
        d = d + s["addend"].float()
    return d.to(torch.bfloat16)


def _own(s):
    from block_scaled_fp8_route_gb300 import ops
    c = s["case"]
    if c["op"] == "gate":
        ids, weights = ops.gate(s["logits"], c["kr"], score=c["score"], bias=s["bias"], groups=c["groups"],
                                kept_groups=c["kept"], group_score=c["group_score"], renormalise=c["renormalise"],
                                scale=c["scale"], topk_ids=s["ids"], topk_weights=s["weights"])
        return {"ids": ids, "weights": weights}
    if c["op"] == "swiglu":
        q, sf = ops.swiglu_quantise(s["y"], rows=s["rows"], q=s["q"], sf=s["sf"])
        return {"q": q.view(torch.float8_e4m3fn), "sf": sf[:, :s["y"].shape[0]]}
    return ops.dense_gemm(s["a"], s["sfa"], s["b"], s["sfb"], c["N"], addend=s["addend"], d=s["d"], flags=ops.B_TILED)


def run(state):
    if own:
        return _own(state)
    return {"gate": _plain_gate, "swiglu": _plain_swiglu, "dense": _plain_dense}[state["case"]["op"]](state)


# ----------------------------------------------------------------------------- 64 bits
def _exact_gate(s):
    c = s["case"]
    T, E, G, kr = c["T"], c["E"], c["groups"], c["kr"]
    l = s["logits"].double().cpu().numpy()
    b = None if s["bias"] is None else s["bias"].double().cpu().numpy()
    off = np.isneginf(l) | np.isnan(l)
    with np.errstate(all="ignore"):
        if c["score"] == "sigmoid":
            p = 1 / (1 + np.exp(-l))
        else:
            top = np.where(off, -1e300, l).max(1, keepdims=True)
            p = np.exp(l - top)
            p[off] = 0
            p = p / np.maximum(p.sum(1, keepdims=True), 1e-300)
    p[off] = 0
    value = p + b if b is not None else p
    key = np.where(off, -np.inf, l if b is None else value)
    if G > 1:
        size = E // G
        if c["group_score"] == "max":
            gs = key.reshape(T, G, size).max(2)
        else:
            v = np.sort(np.where(off, -np.inf, value).reshape(T, G, size), axis=2)
            second = v[:, :, -2] if size > 1 else np.zeros((T, G))
            gs = v[:, :, -1] + np.where(np.isfinite(second), second, 0)
        lost = np.argsort(-gs, axis=1, kind="stable")[:, c["kept"]:]
        dropped = np.zeros((T, G), bool)
        np.put_along_axis(dropped, lost, True, 1)
        key[np.repeat(dropped, size, axis=1)] = -np.inf
    ids = np.argsort(-key, axis=1, kind="stable")[:, :kr]
    none = np.isneginf(np.take_along_axis(key, ids, 1))
    w = np.where(none, 0.0, np.take_along_axis(p, ids, 1))
    if c["renormalise"]:
        w = w / np.where(w.sum(1, keepdims=True) > 0, w.sum(1, keepdims=True), 1.0)
    return {"ids": np.where(none, -1, ids).astype(np.int32), "weights": w * c["scale"]}


def _exact_swiglu(s):
    K, R = s["case"]["K"], s["y"].shape[0]
    codes = torch.arange(127, device=DEV, dtype=torch.float64)        # non-negative E4M3 values, in order
    field, frac = torch.div(codes, 8, rounding_mode="floor"), codes % 8
    values = torch.where(field > 0, (1 + frac / 8) * 2.0 ** (field - 7), frac * 2.0 ** -9)
    half = (values[1:] + values[:-1]) / 2
    out = torch.zeros(R, _padded(K), dtype=torch.float64, device=DEV)
    sf = torch.zeros(s["sf"].shape[0], R, dtype=torch.int64, device=DEV)
    for lo in range(0, R, 8192):                                      # a slice of rows at a time
        y = s["y"][lo:lo + 8192].double()
        h = y[:, K:] * y[:, :K] * torch.sigmoid(y[:, :K])
        n = h.shape[0]
        keep = torch.ones(n, dtype=torch.bool, device=DEV)
        if s["rows"] is not None:
            token, used = s["rows"]
            keep = (token[lo:lo + n] >= 0) & (torch.arange(lo, lo + n, device=DEV) < used)
            h[~keep] = 0
        full = torch.zeros(n, _padded(K), dtype=torch.float64, device=DEV)
        full[:, :K] = h
        blocks = full.view(n, -1, 128)
        amax = blocks.abs().amax(2)
        e = torch.where(amax > 0, torch.ceil(torch.log2(amax / 448)), 0.0)
        v = blocks / 2.0 ** e.unsqueeze(2)
        mag = v.abs().contiguous()
        up, down = torch.bucketize(mag, half, right=True), torch.bucketize(mag, half, right=False)
        near = torch.where((up != down) & (down % 2 == 1), up, down)      # a tie goes to the even code
        out[lo:lo + n] = (torch.copysign(values[near], v)).view(n, -1)
        byte = e.long() + 127
        byte = torch.nn.functional.pad(byte, (0, sf.shape[0] * 4 - byte.shape[1]), value=127).view(n, -1, 4)
        word = byte[..., 0] + (byte[..., 1] << 8) + (byte[..., 2] << 16) + (byte[..., 3] << 24)
        word = torch.where(word >= 1 << 31, word - (1 << 32), word)
        sf[:, lo:lo + n] = torch.where(keep, word.t(), 0)
    return {"q": out, "sf": sf.int()}


def _exact_dense(s):
    c = s["case"]
    M, N, K = c["M"], c["N"], c["K"]
    codes = torch.arange(256, device=DEV)
    field, frac = (codes >> 3) & 15, (codes & 7).double()
    table = torch.where(field > 0, (1 + frac / 8) * 2.0 ** (field - 7).double(), frac * 2.0 ** -9)
    table = torch.where(codes >= 128, -table, table)

    def scales(sf, rows):
        by = sf.cpu().numpy().view(np.uint8).reshape(sf.shape[0], sf.shape[1], 4)[:, :rows]
        by = by.transpose(1, 0, 2).reshape(rows, -1)[:, :K // 128].astype(np.float64)
        return torch.from_numpy(np.repeat(np.exp2(by - 127), 128, axis=1)).to(DEV)

    n = torch.arange(N, device=DEV).view(N, 1)
    k = torch.arange(K, device=DEV).view(1, K)
    at = ((n // 128) * (K // 128) + k // 128) * 16384 + (n % 128) * 128 + k % 128
    b = table[s["b"].view(-1)[at].long()] * scales(s["sfb"], N)
    a = table[s["a"].long()] * scales(s["sfa"], M)
    d = torch.matmul(a, b.T)
    return d if s["addend"] is None else d + s["addend"].double()


def exact(case, seed):
    s = prepare(case, seed)
    return {"gate": _exact_gate, "swiglu": _exact_swiglu, "dense": _exact_dense}[case["op"]](s)
