"""64-bit CPU oracle of the logits' penalties, biases and masks and of the token
counts, from their definitions.  Shares no code with the GPU path."""
from __future__ import annotations

import numpy as np

U = 2.0 ** -24          # half a step of fp32, relative


def unpack(words, V):
    """Truth values [.., V] of packed int32 words."""
    w = np.asarray(words).astype(np.int64) & 0xFFFFFFFF
    return ((w[..., None] >> np.arange(32)) & 1).reshape(*w.shape[:-1], -1)[..., :V].astype(bool)


def pack(bits):
    """int32 words of truth values [.., V]."""
    V = bits.shape[-1]
    b = np.zeros((*bits.shape[:-1], (V + 31) // 32 * 32), dtype=np.int64)
    b[..., :V] = bits
    w = (b.reshape(*bits.shape[:-1], -1, 32) << np.arange(32)).sum(-1)
    return np.where(w >= 2 ** 31, w - 2 ** 32, w).astype(np.int32)


def count_tokens(tokens, lens, V, counts, seen, reset, prompt):
    """(counts, seen as truth values) after tokens[s][:lens[s]]."""
    counts, seen = counts.copy(), seen.copy()
    for s, m in enumerate(lens):
        if reset:
            counts[s], seen[s] = 0, False
        for t in tokens[s][:m]:
            seen[s][t] = True
            if not prompt:
                counts[s][t] += 1
    return counts, seen


def process_row(x, bias, seen, counts, path_tokens, repetition, frequency, presence, allowed,
                masked_value, literal32=False):
    """One row: (values, how far fp32 may be off).  bias: {token: value};
    path_tokens: the drafted tokens on the row's path.  literal32: each
    operation in fp32, rounded once."""
    f = np.float32 if literal32 else np.float64
    x = x.astype(f)
    err = np.zeros(len(x))
    for t, b in bias.items():
        x[t] = x[t] + f(b)
        err[t] = U * abs(float(x[t]))
    met, c = seen.copy(), counts.astype(np.int64) * seen
    for t in path_tokens:
        met[t] = True
        c[t] += 1
    r, fr, pr = f(repetition), f(frequency), f(presence)
    i = np.nonzero(met)[0]
    y, e = x[i], err[i]
    pos = y > 0
    y = np.where(pos, y * (f(1) / r) if literal32 else y / r, y * r).astype(f)
    # the reciprocal's rounding and the product's
    e = np.where(pos, e / float(r) + U * np.abs(y), e * float(r)) + U * np.abs(y)
    p = (fr * c[i].astype(f)).astype(f)
    e = e + U * np.abs(p)
    p = np.where(c[i] > 0, p + pr, p).astype(f)
    e = e + U * np.abs(p)
    y = (y - p).astype(f)
    e = e + U * np.abs(y)
    x[i], err[i] = y, e
    if allowed is not None:
        x[~allowed] = np.float32(masked_value)          # an fp32 argument
        err[~allowed] = 0.0
    return x, err * (1 + 2.0 ** -20)
