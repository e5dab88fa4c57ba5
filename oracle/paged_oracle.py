"""64-bit CPU oracle of the paged-cache operators, from their definitions.

Shares no code with the GPU path.  Tensors are numpy float64 arrays holding
the 16-bit values the kernels read; loops over sequences, tokens and heads.
"""
from __future__ import annotations

import numpy as np


def rope_frequencies(rot_dim, base=10000.0, scaling="plain", factor=1.0, original_len=0.0,
                     low=1.0, high=32.0):
    """(radians a position of each pair, factor of the rotated rows)."""
    c = np.arange(rot_dim // 2)
    if scaling == "base":
        base = base * factor ** (rot_dim / (rot_dim - 2))
    f = base ** (-2.0 * c / rot_dim)
    if scaling == "linear":
        return f / factor, 1.0
    if scaling == "wavelength":
        turns = original_len * f / (2 * np.pi)
        out = np.empty_like(f)
        for i, r in enumerate(turns):
            if r > high:
                out[i] = f[i]
            elif r < low:
                out[i] = f[i] / factor
            else:
                w = (r - low) / (high - low)
                out[i] = (1 - w) * f[i] / factor + w * f[i]
        return out, 1.0
    if scaling == "ramp":
        def index(turns):
            return rot_dim * np.log(original_len / (turns * 2 * np.pi)) / (2 * np.log(base))
        first = max(np.floor(index(high)), 0)
        last = min(np.ceil(index(low)), rot_dim - 1)
        w = np.clip((c - first) / max(last - first, 0.001), 0, 1)
        return f * (1 - w) + f / factor * w, 0.1 * np.log(factor) + 1.0
    return f, 1.0


def rotate_row(x, pos, freqs, rope_scale, interleaved):
    """x [..., d] at one position; returns the rotated row."""
    r = 2 * len(freqs)
    y = x.copy()
    cos, sin = np.cos(pos * freqs) * rope_scale, np.sin(pos * freqs) * rope_scale
    if interleaved:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        y[..., 0:r:2], y[..., 1:r:2] = a * cos - b * sin, b * cos + a * sin
    else:
        a, b = x[..., :r // 2], x[..., r // 2:r]
        y[..., :r // 2], y[..., r // 2:r] = a * cos - b * sin, b * cos + a * sin
    return y


def token_rows(cu_q, seq_lens):
    """(token, sequence, row) of every token that has a row."""
    out = []
    for s in range(len(seq_lens)):
        ql = cu_q[s + 1] - cu_q[s]
        for i in range(ql):
            out.append((cu_q[s] + i, s, seq_lens[s] - ql + i))
    return out


def sequence_rows(pages, table_row, length, kv):
    """Rows [length, d] of one sequence and KV head, in order."""
    ps = pages.shape[2]
    need = (length + ps - 1) // ps
    if need == 0:
        return np.zeros((0, pages.shape[3]))
    return np.concatenate([pages[p, kv] for p in table_row[:need]])[:length]


def softmax_rows(q, k, v, see):
    """One query over keys k [L, d] where see [L]: (o, lse, sum p |v|, largest
    sum |q k| / sqrt(d)); o = 0 and lse = -inf when nothing is seen."""
    d = q.shape[0]
    if not see.any():
        return np.zeros(d), -np.inf, np.zeros(d), 0.0
    ks, vs = k[see], v[see]
    x = ks @ q / np.sqrt(d)
    m = x.max()
    p = np.exp(x - m)
    z = p.sum()
    p /= z
    return p @ vs, m + np.log(z), p @ np.abs(vs), (np.abs(ks) @ np.abs(q)).max() / np.sqrt(d)


def attention(q, k_pages, v_pages, cu_q, seq_lens, table, pages=None, counts=None):
    """(o [n, Hq, d], lse [n, Hq], sum p |v|, largest sum |q k| / sqrt(d) [n, Hq]) in 64 bits;
    tokens of no sequence stay NaN.  pages, counts: the sparse form."""
    n, Hq, d = q.shape
    Hkv, ps = k_pages.shape[1], k_pages.shape[2]
    G = Hq // Hkv
    o, av = np.full((n, Hq, d), np.nan), np.full((n, Hq, d), np.nan)
    lse, aq = np.full((n, Hq), np.nan), np.full((n, Hq), np.nan)
    rows = {}
    for t, s, p in token_rows(cu_q, seq_lens):
        for kv in range(Hkv):
            if (s, kv) not in rows:
                rows[s, kv] = (sequence_rows(k_pages, table[s], seq_lens[s], kv),
                               sequence_rows(v_pages, table[s], seq_lens[s], kv))
            k, v = rows[s, kv]
            key = np.arange(len(k))
            see = key <= p
            if pages is not None:
                chosen = set(int(x) for x in pages[t, kv, :counts[t, kv]])
                see &= np.isin(key // ps, list(chosen))
            for h in range(kv * G, kv * G + G):
                o[t, h], lse[t, h], av[t, h], aq[t, h] = softmax_rows(q[t, h], k, v, see)
    return o, lse, av, aq


def select_pages(q, key_min, key_max, cu_q, seq_lens, table, ps, n_top, n_sink, n_recent):
    """(pages [n, Hkv, N], counts [n, Hkv]); tokens of no sequence hold -7."""
    n, Hq, d = q.shape
    Hkv = key_min.shape[1]
    G = Hq // Hkv
    N = n_sink + n_top + n_recent
    pages = np.full((n, Hkv, N), -7, dtype=np.int32)
    counts = np.full((n, Hkv), -7, dtype=np.int32)
    for t, s, p in token_rows(cu_q, seq_lens):
        vis = 0 if p < 0 else p // ps + 1
        for kv in range(Hkv):
            if vis <= N:
                kept = list(range(vis))
            else:
                score = {}
                for j in range(n_sink, vis - n_recent):
                    mn, mx = key_min[table[s][j], kv], key_max[table[s][j], kv]
                    qs = q[t, kv * G:(kv + 1) * G]
                    with np.errstate(all="ignore"):
                        x = np.float32(np.maximum(qs * mn, qs * mx).sum())
                    good = np.isfinite(x) and np.isfinite(mn).all() and np.isfinite(mx).all()
                    score[j] = x if good else np.float32(-np.inf)
                best = sorted(score, key=lambda j: (-score[j], j))[:n_top]
                kept = list(range(n_sink)) + sorted(best) + list(range(vis - n_recent, vis))
            counts[t, kv] = len(kept)
            pages[t, kv] = kept + [-1] * (N - len(kept))
    return pages, counts


def root_paths(parents):
    """Each node's ancestors and itself, root first; the first node is the root."""
    paths = []
    for i, p in enumerate(parents):
        paths.append((paths[p] if i else []) + [i])
    return paths


def tree_attention(q, k_pages, v_pages, cu_q, seq_lens, table, parents):
    """attention() with each sequence's tokens as the nodes of a tree: a node sees
    the rows in front of the tree, its ancestors' and its own."""
    n, Hq, d = q.shape
    Hkv = k_pages.shape[1]
    G = Hq // Hkv
    o, av = np.full((n, Hq, d), np.nan), np.full((n, Hq, d), np.nan)
    lse, aq = np.full((n, Hq), np.nan), np.full((n, Hq), np.nan)
    for s, kl in enumerate(seq_lens):
        t0, ql = cu_q[s], cu_q[s + 1] - cu_q[s]
        if ql == 0:
            continue
        paths = root_paths([int(p) for p in parents[t0:t0 + ql]])
        see = np.tile(np.arange(kl) < kl - ql, (ql, 1))
        for i in range(ql):
            see[i, [kl - ql + a for a in paths[i] if kl - ql + a >= 0]] = True
        see = np.repeat(see, G, axis=0)                     # rows (node, head of the group)
        none = ~see.any(1)
        for kv in range(Hkv):
            k = sequence_rows(k_pages, table[s], kl, kv)
            v = sequence_rows(v_pages, table[s], kl, kv)
            hs = slice(kv * G, kv * G + G)
            x = q[t0:t0 + ql, hs].reshape(-1, d)
            at = np.where(see, x @ k.T / np.sqrt(d), -np.inf)
            top = np.where(none, 0.0, at.max(1, initial=-np.inf))
            p = np.exp(at - top[:, None])
            z = p.sum(1)
            p /= np.where(none, 1.0, z)[:, None]
            size = np.where(see, np.abs(x) @ np.abs(k).T, 0.0).max(1, initial=0.0) / np.sqrt(d)
            with np.errstate(divide="ignore"):
                total = np.where(none, -np.inf, top + np.log(z))
            o[t0:t0 + ql, hs] = (p @ v).reshape(ql, G, d)
            av[t0:t0 + ql, hs] = (p @ np.abs(v)).reshape(ql, G, d)
            lse[t0:t0 + ql, hs] = total.reshape(ql, G)
            aq[t0:t0 + ql, hs] = size.reshape(ql, G)
    return o, lse, av, aq


def kv_commit(k_pages, v_pages, key_min, key_max, cu_q, seq_lens, table, path, n_path):
    """One layer's (k, v, key_min, key_max, new lengths) after the accepted rows'
    move; key_min, key_max None: no bounds.  Arrays are copied."""
    k, v = k_pages.copy(), v_pages.copy()
    mn, mx = (None, None) if key_min is None else (key_min.copy(), key_max.copy())
    ps = k.shape[2]
    new = []
    for s, kl in enumerate(seq_lens):
        ql = cu_q[s + 1] - cu_q[s]
        if ql == 0:
            new.append(kl)
            continue
        L, m = kl - ql, n_path[s]

        def at(r):
            return table[s][r // ps], r % ps

        src = [at(L + path[s][t]) for t in range(1, m)]
        rows = [(k_pages[p, :, r], v_pages[p, :, r]) for p, r in src]
        for t in range(1, m):
            p, r = at(L + t)
            k[p, :, r], v[p, :, r] = rows[t - 1]
        new.append(L + m)
        if mn is None:
            continue
        for pg in range(L // ps, (L + m - 1) // ps + 1):
            held = [k[table[s][pg], :, r - pg * ps] for r in range(max(L, pg * ps), min(L + m, (pg + 1) * ps))]
            if pg * ps < L:
                held += [mn[table[s][pg]], mx[table[s][pg]]]
            mn[table[s][pg]] = np.min(held, axis=0)
            mx[table[s][pg]] = np.max(held, axis=0)
    return k, v, mn, mx, new
