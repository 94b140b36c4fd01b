"""A layer in which the terms that ``few_token_moe`` splits h into can be told apart from their sum."""

import numpy as np
import torch


def cancelling(T, E=3, K=128, I=128, seed=0):
    """(x, ids, weights, w13, w2) whose z is 0 in exact arithmetic: gate rows 2 j and 2 j + 1 are equal, up row 2 j + 1 is three
    times row 2 j, and each row of w2 takes 3 h of the first and -1 of the second.  What is left of z is the error of
    each h on its own, 3 err(h) - err(3 h), neither averaged over a long sum nor below z's own rounding.  All weights are
    small powers of two or three times one, exact in bf16 and in E4M3."""
    r = np.random.default_rng(seed)
    w13, w2 = np.zeros((E, 2 * I, K), np.float32), np.zeros((E, K, I), np.float32)
    for e in range(E):
        for j in range(0, I, 2):
            for base, sizes in ((0, (0.5, 1.0)), (I, (0.5, 1.0, 2.0))):
                at = r.permutation(K)[:4]
                w13[e, base + j, at] = r.choice(sizes, 4) * r.choice((-1, 1), 4)
                w13[e, base + j + 1] = w13[e, base + j] * (1 if base == 0 else 3)
        for n in range(K):
            j = 2 * (n % (I // 2))
            w2[e, n, j], w2[e, n, j + 1] = 3, -1
    bf16 = lambda a: torch.from_numpy(np.float32(a)).to(torch.bfloat16)  # noqa: E731
    ids = torch.from_numpy(r.integers(0, E, (T, 1)).astype(np.int32))
    weights = torch.from_numpy(r.uniform(0.3, 1.0, (T, 1)).astype(np.float32))
    return bf16(r.standard_normal((T, K))), ids, weights, bf16(w13), bf16(w2)
