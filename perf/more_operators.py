"""Cases for the whole mixture-of-experts layer of a few tokens (``moe``) and the unquantised matrix product with bias,
activation and residual in its epilogue (``linear``), which among others computes the router's logits.

``run`` computes them with elementary torch operations in float32 (``own`` false) or calls the package's
operators (``own`` true); ``exact`` computes them in 64 bits from their definitions.
"""

import math

import torch

own = False

DEV = "cuda"


# ----------------------------------------------------------------------------- cases
def listed():
    return [
        # the tiny workload's layer, three tokens: nothing but latency
        dict(name="moe_tiny", op="moe", T=3, E=8, kr=2, K=256, I=128, S=0, weights="fp8", pad=0, addend=False),
        # one sequence being decoded: the chosen experts' weights stream once for a single token
        dict(name="moe_one_token", op="moe", T=1, E=128, kr=8, K=4096, I=1536, S=0, weights="fp8", pad=0,
             addend=False),
        # a few sequences through a wide layer with an always-active expert, added to the residual stream
        dict(name="moe_five_tokens", op="moe", T=5, E=256, kr=8, K=7168, I=2048, S=2048, weights="fp8", pad=0,
             addend=True),
        # unquantised weights, an odd number of 128-blocks, an always-active expert twice as wide
        dict(name="moe_bf16", op="moe", T=7, E=64, kr=6, K=2048, I=1408, S=2816, weights="bf16", pad=0, addend=False),
        # a decode batch padded to a fixed graph size: the padding rows choose no expert
        dict(name="moe_padded_batch", op="moe", T=16, E=128, kr=8, K=4096, I=1536, S=0, weights="fp8", pad=3,
             addend=False),
        # the largest batch of this form: most experts are chosen by someone
        dict(name="moe_full_batch", op="moe", T=32, E=128, kr=8, K=4096, I=1536, S=0, weights="fp8", pad=0,
             addend=True),
        # small ragged product, everything in the epilogue
        dict(name="linear_small", op="linear", T=3, N=130, K=264, dtype="bf16", out="bf16", bias=True, act="silu",
             residual=True),
        # router logits of one decoded token
        dict(name="linear_router_token", op="linear", T=1, N=256, K=7168, dtype="bf16", out="f32", bias=False,
             act="none", residual=False),
        # output projection of a ragged decode batch, added to the residual stream
        dict(name="linear_projection", op="linear", T=37, N=7168, K=4096, dtype="bf16", out="bf16", bias=False,
             act="none", residual=True),
        # router logits of a large prefill batch: every token is read once for a narrow output
        dict(name="linear_router_batch", op="linear", T=8192, N=256, K=7168, dtype="bf16", out="f32", bias=True,
             act="none", residual=False),
        # feed-forward product of a chunk in half precision, ragged in both directions
        dict(name="linear_chunk", op="linear", T=777, N=4100, K=1416, dtype="f16", out="f16", bias=True, act="gelu",
             residual=False),
        # projection of a large prefill batch with bias and residual
        dict(name="linear_large", op="linear", T=8192, N=7168, K=4096, dtype="bf16", out="bf16", bias=True,
             act="none", residual=True),
    ]


ACTS = ["none", "relu", "silu", "gelu", "gelu_tanh", "sigmoid"]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _most(op):
    got = [c for c in listed() if c["op"] == op]
    return max(work(c)["bytes" if op == "moe" else "flops"] for c in got)


def draw(rng):
    if rng.random() < 0.5:
        weights = rng.choice(["fp8", "fp8", "bf16"])
        while True:
            T = _log_int(rng, 1, 32)
            E = rng.choice([4, 8, 16, 40, 64, 128, 160, 256])
            c = dict(op="moe", T=T, E=E, kr=rng.randint(1, min(8, E)), K=128 * _log_int(rng, 1, 56),
                     I=128 * _log_int(rng, 1, 16), S=128 * _log_int(rng, 1, 20) if rng.random() < 0.4 else 0,
                     weights=weights, pad=rng.randint(0, T // 2) if rng.random() < 0.4 else 0,
                     addend=rng.random() < 0.4)
            size = 1 if weights == "fp8" else 2
            expert = 3 * c["K"] * c["I"]
            if work(c)["bytes"] <= _most("moe") and T * c["kr"] * expert <= 32 * 8 * 3 * 4096 * 1536 and \
                    E * expert * size < 12e9:
                return c
    while True:
        dtype = rng.choice(["bf16", "bf16", "f16"])
        c = dict(op="linear", T=_log_int(rng, 1, 8192), N=_log_int(rng, 8, 8192), K=8 * _log_int(rng, 4, 1024),
                 dtype=dtype, out=rng.choice([dtype, dtype, "f32"]), bias=rng.random() < 0.5, act=rng.choice(ACTS),
                 residual=rng.random() < 0.5)
        if work(c)["flops"] <= _most("linear"):
            return c


def work(case):
    if case["op"] == "moe":
        T, E, kr, K, I, S = (case[k] for k in ("T", "E", "kr", "K", "I", "S"))
        live = T - case["pad"]
        chosen = E * (1 - (1 - kr / E) ** live)          # experts that some token chooses, on average
        size = 1 if case["weights"] == "fp8" else 2
        scales = 4 / 512 if case["weights"] == "fp8" else 0
        return {"bytes": (chosen * I + S) * 3 * K * (size + scales) + T * K * (6 if case["addend"] else 4) + T * kr * 8,
                "flops": 6 * K * (live * kr * I + T * S)}
    T, N, K = case["T"], case["N"], case["K"]
    out = 4 if case["out"] == "f32" else 2
    return {"bytes": 2 * K * (T + N) + T * N * out * (2 if case["residual"] else 1) + (4 * N if case["bias"] else 0),
            "flops": 2 * T * N * K}


# ----------------------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _fp8_weights(g, E, N, K):
    """Random weights as a program keeps them: E4M3 codes, 128 x 128 blocks contiguous ([E, N, K] bytes), and one
    packed word of UE8M0 scale bytes per row and 512 K ([E, ceil(K / 512), N])."""
    blocks = E * (N // 128) * (K // 128)
    codes = torch.empty(blocks, 128, 128, dtype=torch.uint8, device=DEV)
    exps = torch.empty(blocks, dtype=torch.int64, device=DEV)
    for lo in range(0, blocks, 16384):
        n = min(16384, blocks - lo)
        w = torch.randn(n, 128, 128, device=DEV, generator=g)
        # blocks differ in size, as rows of a trained matrix do
        w *= 0.02 * torch.exp2(torch.randint(-1, 2, (n, 1, 1), device=DEV, generator=g))
        amax = w.abs().amax((1, 2))
        m, ex = torch.frexp(amax)
        e = ex - 9 + (m > 0.875).int()                   # the least e with amax <= 448 * 2**e
        codes[lo:lo + n] = (w * torch.ldexp(torch.ones_like(amax), -e).view(n, 1, 1)).to(torch.float8_e4m3fn).view(
            torch.uint8)
        exps[lo:lo + n] = e
    nkb, words = K // 128, (K // 128 + 3) // 4
    b = torch.full((E, N // 128, words * 4), 127, dtype=torch.int64, device=DEV)
    b[:, :, :nkb] = exps.view(E, N // 128, nkb) + 127
    b = b.view(E, N // 128, words, 4)
    w = b[..., 0] | b[..., 1] << 8 | b[..., 2] << 16 | b[..., 3] << 24
    w = torch.where(w >= 1 << 31, w - (1 << 32), w).int()
    return codes.view(E, N, K), w.permute(0, 2, 1).repeat_interleave(128, 2).contiguous()


def _bf16_weights(g, E, N, K):
    """Random bf16 weights in boxes of 128 rows x 64 values, given as bytes [E, N, 2 K]; they have no scales."""
    w = torch.empty(E, N, K, dtype=torch.bfloat16, device=DEV)
    step = max(1, (1 << 28) // (N * K))
    for lo in range(0, E, step):
        n = min(step, E - lo)
        w[lo:lo + n] = 0.02 * torch.randn(n, N, K, device=DEV, generator=g)
    return w.view(torch.uint8), None


def _prepare_moe(case, seed):
    g = _gen(seed)
    T, E, kr, K, I, S = (case[k] for k in ("T", "E", "kr", "K", "I", "S"))
    make = _fp8_weights if case["weights"] == "fp8" else _bf16_weights
    w13, sf13 = make(g, E, 2 * I, K)
    w2, sf2 = make(g, E, K, I)
    shared = None
    if S:
        shared = make(g, 1, 2 * S, K) + make(g, 1, K, S)
        shared = tuple(None if t is None else t[0] for t in shared)
    x = torch.randn(T, K, device=DEV, generator=g)
    x[:, torch.rand(K, device=DEV, generator=g) < 0.002] *= 30.0          # outlier channels
    # each token's kr distinct experts, the largest of its router scores first; softmax weights over them
    scores, ids = torch.randn(T, E, device=DEV, generator=g).topk(kr, dim=1)
    weights = torch.softmax(scores, 1)
    if case["pad"]:
        ids[T - case["pad"]:] = -1
        weights[T - case["pad"]:] = 0.0
    addend = torch.randn(T, K, device=DEV, generator=g).to(torch.bfloat16) if case["addend"] else None
    z = torch.zeros(T, K, dtype=torch.bfloat16, device=DEV)
    return dict(case=case, x=x.to(torch.bfloat16), ids=ids.int().contiguous(), weights=weights.contiguous(), w13=w13,
                sf13=sf13, w2=w2, sf2=sf2, shared=shared, addend=addend, z=z)


TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def _prepare_linear(case, seed):
    g = _gen(seed)
    T, N, K = case["T"], case["N"], case["K"]
    dtype, out = TYPES[case["dtype"]], TYPES[case["out"]]
    x = torch.randn(T, K, device=DEV, generator=g)
    x[torch.rand(T, device=DEV, generator=g) < 0.01] *= 10.0              # outlier tokens
    w = torch.randn(N, K, device=DEV, generator=g) / math.sqrt(K)
    bias = 0.1 * torch.randn(N, device=DEV, generator=g) if case["bias"] else None
    residual = torch.randn(T, N, device=DEV, generator=g).to(out) if case["residual"] else None
    return dict(case=case, x=x.to(dtype), w=w.to(dtype), bias=bias, residual=residual,
                y=torch.zeros(T, N, dtype=out, device=DEV))


def prepare(case, seed):
    return {"moe": _prepare_moe, "linear": _prepare_linear}[case["op"]](case, seed)


# ----------------------------------------------------------------------------- one pass
def _rows(b, sf):
    """Weights [n, N, K] in float32 from boxes of 128 rows x 128 bytes (and their scale words)."""
    n, N, width = b.shape
    b = b.view(n, N // 128, width // 128, 128, 128).transpose(2, 3).reshape(n, N, width)
    if sf is None:
        return b.view(torch.bfloat16).float()
    e = torch.stack([sf & 255, sf >> 8 & 255, sf >> 16 & 255, sf >> 24 & 255], 2) - 127      # [n, words, 4, N]
    e = e.flatten(1, 2)[:, :width // 128].transpose(1, 2)
    scale = torch.ldexp(torch.ones((), device=DEV), e).unsqueeze(3)                          # [n, N, K / 128, 1]
    return (b.view(torch.float8_e4m3fn).float().view(n, N, width // 128, 128) * scale).view(n, N, width)


def _plain_moe(s):
    c = s["case"]
    T, kr = c["T"], c["kr"]
    x = s["x"].float()
    pick = s["ids"].flatten().clamp(min=0).long()
    rows = x.repeat_interleave(kr, 0).unsqueeze(2)                        # one row per choice
    at = [None if t is None else t[pick] for t in (s["sf13"], s["sf2"])]
    g, u = torch.bmm(_rows(s["w13"][pick], at[0]), rows).squeeze(2).chunk(2, 1)
    h = g / (1.0 + torch.exp(-g)) * u
    y = torch.bmm(_rows(s["w2"][pick], at[1]), h.unsqueeze(2)).view(T, kr, -1)
    z = (y * torch.where(s["ids"] >= 0, s["weights"], 0.0).unsqueeze(2)).sum(1)
    if s["shared"] is not None:
        b13, sf13, b2, sf2 = (None if t is None else t.unsqueeze(0) for t in s["shared"])
        g, u = (x @ _rows(b13, sf13)[0].t()).chunk(2, 1)
        z = z + (g / (1.0 + torch.exp(-g)) * u) @ _rows(b2, sf2)[0].t()
    if s["addend"] is not None:
        z = z + s["addend"].float()
    return z.to(torch.bfloat16)


def _plain_act(v, act):
    if act == "relu":
        return v.clamp(min=0.0)
    if act == "silu":
        return v / (1.0 + torch.exp(-v))
    if act == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-v))
    if act == "gelu":
        return 0.5 * v * (1.0 + torch.erf(v * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * v * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (v + 0.044715 * v * v * v)))
    return v


def _plain_linear(s):
    v = s["x"].float() @ s["w"].float().t()
    if s["bias"] is not None:
        v = v + s["bias"]
    v = _plain_act(v, s["case"]["act"])
    if s["residual"] is not None:
        v = v + s["residual"].float()
    return v.to(s["y"].dtype)


def _own(s):
    from block_scaled_fp8_route_gb300 import ops
    c = s["case"]
    if c["op"] == "moe":
        return ops.few_token_moe(s["x"], s["ids"], s["weights"], s["w13"], s["sf13"], s["w2"], s["sf2"],
                                 shared=s["shared"], addend=s["addend"], z=s["z"], flags=ops.B_TILED)
    return ops.linear(s["x"], s["w"], bias=s["bias"], activation=c["act"], residual=s["residual"], out=s["y"])


def run(state):
    if own:
        return _own(state)
    return {"moe": _plain_moe, "linear": _plain_linear}[state["case"]["op"]](state)


# ----------------------------------------------------------------------------- 64 bits
def _table():
    codes = torch.arange(256, device=DEV)
    field, frac = (codes >> 3) & 15, (codes & 7).double()
    value = torch.where(field > 0, (1 + frac / 8) * 2.0 ** (field - 7).double(), frac * 2.0 ** -9)
    return torch.where(codes >= 128, -value, value)


def _wide(b, sf, table):
    """One matrix [N, K] in 64 bits."""
    N, width = b.shape
    per = 128 if sf is not None else 64
    flat = b.reshape(-1).to(torch.int32)
    n = torch.arange(N, device=DEV).view(N, 1)
    if sf is None:
        k = torch.arange(width // 2, device=DEV).view(1, -1)
        at = ((n // 128) * (width // 128) + k // per) * 16384 + (n % 128) * 128 + 2 * (k % per)
        bits = flat[at + 1] << 24 | flat[at] << 16
        return bits.view(torch.float32).double()
    k = torch.arange(width, device=DEV).view(1, -1)
    at = ((n // 128) * (width // 128) + k // per) * 16384 + (n % 128) * 128 + k % per
    byte = (sf[k // 512, n] >> (8 * (k // 128 % 4)).int()) & 255
    return table[flat[at].long()] * torch.pow(2.0, byte.double() - 127)


def _exact_moe(s):
    c, table = s["case"], _table()
    x, I, S = s["x"].double(), c["I"], c["S"]
    z = torch.zeros(c["T"], c["K"], dtype=torch.float64, device=DEV)

    def expert(rows, b13, sf13, b2, sf2, width):
        y = torch.matmul(rows, _wide(b13, sf13, table).T)
        h = y[:, :width] * torch.sigmoid(y[:, :width]) * y[:, width:]
        return torch.matmul(h, _wide(b2, sf2, table).T)

    for e in sorted(set(s["ids"].flatten().tolist()) - {-1}):
        share = torch.where(s["ids"] == e, s["weights"].double(), 0.0).sum(1)
        t = (s["ids"] == e).any(1).nonzero().flatten()
        sf13, sf2 = (None, None) if s["sf13"] is None else (s["sf13"][e], s["sf2"][e])
        z[t] += share[t].unsqueeze(1) * expert(x[t], s["w13"][e], sf13, s["w2"][e], sf2, I)
    if S:
        z += expert(x, *s["shared"], S)
    return z if s["addend"] is None else z + s["addend"].double()


def _exact_linear(s):
    v = torch.matmul(s["x"].double(), s["w"].double().T)
    if s["bias"] is not None:
        v += s["bias"].double()
    act = s["case"]["act"]
    if act == "relu":
        v = torch.where(v > 0, v, 0.0)
    elif act in ("silu", "sigmoid"):
        p = torch.special.expit(v)
        v = v * p if act == "silu" else p
    elif act == "gelu":
        v = v * torch.special.ndtr(v)
    elif act == "gelu_tanh":
        v = v * torch.special.expit(2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3))
    return v if s["residual"] is None else v + s["residual"].double()


def exact(case, seed):
    s = prepare(case, seed)
    return {"moe": _exact_moe, "linear": _exact_linear}[case["op"]](s)
