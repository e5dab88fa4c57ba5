"""Measured cases of the paged-cache operators.

Four operators work on one paged K/V cache ([n_pages, Hkv, page, d]; a
sequence's rows sit in the pages its row of the page table names): the rotary
append of new tokens, attention of new tokens over the pages, the choice of
pages by a bound on their scores, and attention over the chosen pages.  Each
case holds plain numbers; `run` makes one pass, in elementary torch operations
or (`own`) through the library's calls; `exact` is the definition in 64 bits.
"""
import math
import random

import numpy as np
import torch

own = False

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # next token of a few streams, 1.5B-shaped layer: latency only
        dict(name="append_decode", op="append", n_seq=4, q=1, kv=32768, Hq=12, Hkv=2, d=128,
             page=16, dtype="bf16", rot=128, inter=False, factor=1.0, tree=False, bounds=True,
             ragged=True, shape=1),
        # a 64-node draft tree at 100K tokens, 14B-shaped layer, stretched rotation
        dict(name="append_tree", op="append", n_seq=1, q=64, kv=102400, Hq=40, Hkv=8, d=128,
             page=64, dtype="bf16", rot=128, inter=False, factor=4.0, tree=True, bounds=True,
             ragged=False, shape=2),
        # a batch of prompts entering the cache, 7B MHA-shaped layer, half of the head rotated
        dict(name="append_prompts", op="append", n_seq=6, q=2048, kv=4096, Hq=32, Hkv=32, d=128,
             page=128, dtype="fp16", rot=64, inter=True, factor=1.0, tree=False, bounds=False,
             ragged=True, shape=3),
        # next token of three short streams, tiny layer: the smallest attention call
        dict(name="decode_tiny", op="attend", n_seq=3, q=1, kv=4096, Hq=4, Hkv=1, d=64, page=16,
             dtype="bf16", ragged=True, shape=4),
        # next token of one stream at 100K tokens, 8B-shaped layer
        dict(name="decode_100k", op="attend", n_seq=1, q=1, kv=102397, Hq=32, Hkv=8, d=128,
             page=64, dtype="bf16", ragged=False, shape=5),
        # next token of a ragged batch, 14B-shaped layer (five query heads a KV head)
        dict(name="decode_batch", op="attend", n_seq=16, q=1, kv=32768, Hq=40, Hkv=8, d=128,
             page=32, dtype="fp16", ragged=True, shape=6),
        # a prompt chunk over a 32K cache, 1.5B-shaped layer
        dict(name="chunk_32k", op="attend", n_seq=1, q=2048, kv=32768, Hq=12, Hkv=2, d=128,
             page=16, dtype="bf16", ragged=False, shape=7),
        # prompts, chunks and single tokens in one call, small heads
        dict(name="chunk_mixed", op="attend", n_seq=9, q=1500, kv=6000, Hq=16, Hkv=4, d=64,
             page=32, dtype="fp16", ragged=True, shape=8),
        # a prompt chunk at 100K tokens, 8B-shaped layer: the largest
        dict(name="chunk_100k", op="attend", n_seq=1, q=2048, kv=102400, Hq=32, Hkv=8, d=128,
             page=64, dtype="bf16", ragged=False, shape=9),
        # pages chosen for a batch of long streams, 8B-shaped layer
        dict(name="select_batch", op="select", n_seq=16, q=1, kv=102400, Hq=32, Hkv=8, d=128,
             page=32, dtype="bf16", n_top=128, n_sink=1, n_recent=2, ragged=True, shape=10),
        # attention over chosen pages (4096 tokens of up to 100K), 14B-shaped layer
        dict(name="selected_batch", op="selected", n_seq=8, q=1, kv=102400, Hq=40, Hkv=8, d=128,
             page=64, dtype="bf16", n_top=61, n_sink=1, n_recent=2, ragged=True, shape=11),
        # choice and attention for one stream, 1.5B-shaped layer: the sparse step's latency
        dict(name="sparse_step", op="sparse", n_seq=1, q=1, kv=32768, Hq=12, Hkv=2, d=128,
             page=16, dtype="fp16", n_top=128, n_sink=1, n_recent=4, ragged=False, shape=12),
    ]


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "select", "selected", "sparse"])
    heads = rng.choice([(4, 1), (12, 2), (16, 4), (32, 8), (40, 8), (8, 8)])
    log = lambda lo, hi: int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))  # noqa: E731
    c = dict(op=op, Hq=heads[0], Hkv=heads[1], d=rng.choice([64, 128, 128]),
             page=rng.choice([16, 32, 64, 128]), dtype=rng.choice(["bf16", "fp16"]),
             ragged=rng.random() < 0.6, shape=rng.randrange(1 << 30))
    if op == "append":
        c.update(n_seq=log(1, 24), q=log(1, 700), kv=log(1000, 102400),
                 rot=rng.choice([c["d"], c["d"], c["d"] // 2, 16]), inter=rng.random() < 0.4,
                 factor=rng.choice([1.0, 1.0, 4.0, 8.0]), tree=rng.random() < 0.3,
                 bounds=rng.random() < 0.7)
    elif op == "attend":
        q, n_seq = 1 if rng.random() < 0.4 else log(2, 2048), log(1, 16)
        # the batch's cache and its query-key pairs stay below the largest listed ones
        top = min(102400, 300000 // n_seq, int(1.5e8 / (n_seq * q)))
        c.update(n_seq=n_seq, q=q, kv=log(min(max(q, 16), top), top))
    else:
        n_seq = log(1, 16)
        c.update(n_seq=n_seq, q=rng.choice([1, 1, 1, 3]), kv=log(1000, min(102400, 600000 // n_seq)),
                 n_top=log(4, 200), n_sink=rng.randrange(0, 3), n_recent=rng.randrange(1, 5))
    return c


def _lengths(case):
    """New tokens and cache lengths (new tokens included) of every sequence."""
    rng = random.Random(case["shape"])
    n, q, kv = case["n_seq"], case["q"], case["kv"]
    if not case["ragged"]:
        return [q] * n, [max(kv, q)] * n
    ql = [q if q == 1 else rng.choice([q, rng.randint(1, q), rng.randint(1, q)]) for _ in range(n)]
    kl = [max(ql[i], rng.randint(max(1, kv // 8), kv)) for i in range(n)]
    kl[-1] = max(kv, ql[-1])
    if case["op"] == "attend" and q > 1 and n > 2:
        ql[0] = 0                       # a stream with nothing new in this call
        ql[1] = 1                       # and one that decodes
        kl[2] = ql[2]                   # and one whose prompt starts here
    return ql, kl


# ------------------------------------------------------------------ inputs
def _frequencies(rot, factor):
    """Angle per position of each pair; factor > 1 stretches the base."""
    if rot == 0:
        return np.zeros(0)
    base = 10000.0 * (factor ** (rot / (rot - 2)) if factor > 1.0 else 1.0)
    return base ** (-np.arange(0, rot, 2, dtype=np.float64) / rot)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    host = random.Random(seed)
    dt = DT[case["dtype"]]
    Hq, Hkv, d, ps = case["Hq"], case["Hkv"], case["d"], case["page"]
    ql, kl = _lengths(case)
    n = sum(ql)

    def normal(*shape):
        return torch.empty(shape, dtype=dt, device="cuda").normal_(generator=g)

    def ints(x):
        return torch.tensor(x, dtype=torch.int32, device="cuda")

    pages_of = [(x + ps - 1) // ps for x in kl]
    maxp = max(pages_of)
    n_pages = sum(pages_of) + 3
    perm = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    table = torch.zeros((len(kl), maxp), dtype=torch.int32, device="cuda")
    at = 0
    for s, np_ in enumerate(pages_of):
        table[s, :np_] = perm[at:at + np_]
        at += np_
    cu = [0]
    for x in ql:
        cu.append(cu[-1] + x)
    st = dict(case=case, ql=ql, kl=kl, cu=cu, n=n, n_pages=n_pages, cu_q=ints(cu),
              seq_lens=ints(kl), table=table)
    if case["op"] == "append":
        # rows of the layer's fused projection: q, k and v of a token side by side
        st["qkv"] = normal(n, (Hq + 2 * Hkv) * d)
        st["freqs"] = torch.tensor(_frequencies(case["rot"], case["factor"]), dtype=torch.float64,
                                   device="cuda")
        st["scale"] = 0.1 * math.log(case["factor"]) + 1.0
        st["positions"] = None
        if case["tree"]:
            # a tree node stands at its depth behind the committed tokens
            pos = []
            for a, b in zip(ql, kl):
                pos += [b - a + min(i, host.randrange(0, 5)) for i in range(a)]
            st["positions"] = ints(pos)
        st["k_pages"] = normal(n_pages, Hkv, ps, d)
        st["v_pages"] = normal(n_pages, Hkv, ps, d)
        st["bounds"] = None
        if case["bounds"]:
            st["bounds"] = (st["k_pages"].amin(2).contiguous(), st["k_pages"].amax(2).contiguous())
        return st
    st["q"] = normal(n, Hq, d)
    if case["op"] == "select":
        # bounds of pages whose keys are N(0, 1) with a few channels offset
        mid = normal(n_pages, Hkv, d) * 0.5
        mid[:, :, ::16] += 1.0
        half = normal(n_pages, Hkv, d).abs() * 0.4 + 1.5
        st["bounds"] = ((mid - half).contiguous(), (mid + half).contiguous())
        return st
    st["k_pages"] = normal(n_pages, Hkv, ps, d)
    st["v_pages"] = normal(n_pages, Hkv, ps, d)
    # heavy hitters: rows of every fortieth page point along the group's last queries
    for s in range(len(ql)):
        if ql[s] and pages_of[s] > 0:
            hot = table[s, :pages_of[s]][host.randrange(0, 3)::40].long()
            dirn = st["q"][cu[s + 1] - 1].view(Hkv, Hq // Hkv, d).float().mean(1)
            row = host.randrange(ps)
            st["k_pages"][hot, :, row] = (st["k_pages"][hot, :, row].float() + 1.5 * dirn).to(dt)
    if case["op"] in ("sparse", "selected"):
        st["bounds"] = (st["k_pages"].amin(2).contiguous(), st["k_pages"].amax(2).contiguous())
    if case["op"] == "selected":
        # a choice as the page scores make it: sinks, recent pages, any pages between
        N = case["n_top"] + case["n_sink"] + case["n_recent"]
        pages = torch.full((n, Hkv, N), -1, dtype=torch.int32)
        counts = torch.zeros((n, Hkv), dtype=torch.int32)
        gen = torch.Generator().manual_seed(seed)
        for s in range(len(ql)):
            for i in range(ql[s]):
                vis = (kl[s] - ql[s] + i) // ps + 1
                m = min(vis, N)
                for h in range(Hkv):
                    if vis <= N:
                        pick = torch.arange(vis)
                    else:
                        lo, hi = case["n_sink"], vis - case["n_recent"]
                        mid = torch.randperm(hi - lo, generator=gen)[:case["n_top"]] + lo
                        pick = torch.cat([torch.arange(lo), mid.sort().values,
                                          torch.arange(hi, vis)])
                    pages[cu[s] + i, h, :m] = pick.int()
                    counts[cu[s] + i, h] = m
        st["pages"], st["counts"] = pages.cuda(), counts.cuda()
    return st


# ------------------------------------------------------------------ one pass
def run(state):
    if own:
        return _run_own(state)
    op = state["case"]["op"]
    if op == "append":
        return _plain_append(state)
    if op == "attend":
        return _plain_attend(state)
    if op == "select":
        return _plain_select(state)
    if op == "selected":
        return _plain_selected(state, state["pages"], state["counts"])
    pages, counts = _plain_select(state)
    return (pages, counts) + _plain_selected(state, pages, counts)


def _split_qkv(st):
    c = st["case"]
    Hq, Hkv, d = c["Hq"], c["Hkv"], c["d"]
    x = st["qkv"]
    return (x[:, :Hq * d].view(-1, Hq, d), x[:, Hq * d:(Hq + Hkv) * d].view(-1, Hkv, d),
            x[:, (Hq + Hkv) * d:].view(-1, Hkv, d))


def _run_own(st):
    import self_speculative_ultra_gb300 as ts
    c = st["case"]
    op = c["op"]
    if op == "append":
        q, k, v = _split_qkv(st)
        kmin, kmax = st["bounds"] if st["bounds"] else (None, None)
        q_out = ts.ts_paged_rope_append(q, k, v, st["cu_q"], st["seq_lens"], st["table"],
                                        st["k_pages"], st["v_pages"], st["freqs"],
                                        positions=st["positions"], rope_scale=st["scale"],
                                        interleaved=c["inter"], key_min=kmin, key_max=kmax)
        out = (q_out, st["k_pages"], st["v_pages"])
        return out + tuple(st["bounds"]) if st["bounds"] else out
    if op == "attend":
        return ts.ts_paged_attention(st["q"], st["k_pages"], st["v_pages"], st["cu_q"],
                                     st["seq_lens"], st["table"], max_q=max(st["ql"]))
    if op == "select":
        return ts.ts_paged_select_pages(st["q"], st["bounds"][0], st["bounds"][1], st["cu_q"],
                                        st["seq_lens"], st["table"], c["page"], c["n_top"],
                                        c["n_sink"], c["n_recent"])
    if op == "selected":
        return ts.ts_paged_attention_selected(st["q"], st["k_pages"], st["v_pages"], st["cu_q"],
                                              st["seq_lens"], st["table"], st["pages"],
                                              st["counts"])
    pages, counts = ts.ts_paged_select_pages(st["q"], st["bounds"][0], st["bounds"][1], st["cu_q"],
                                             st["seq_lens"], st["table"], c["page"], c["n_top"],
                                             c["n_sink"], c["n_recent"])
    o, lse = ts.ts_paged_attention_selected(st["q"], st["k_pages"], st["v_pages"], st["cu_q"],
                                            st["seq_lens"], st["table"], pages, counts)
    return pages, counts, o, lse


def _plain_append(st):
    c = st["case"]
    ps, rot = c["page"], c["rot"]
    dt = DT[c["dtype"]]
    q, k, v = _split_qkv(st)
    dev = q.device
    cu = st["cu_q"].long()
    seq = torch.repeat_interleave(torch.arange(len(st["ql"]), device=dev), cu[1:] - cu[:-1],
                                  output_size=st["n"])
    slot = st["seq_lens"].long()[seq] - cu[seq + 1] + torch.arange(st["n"], device=dev)
    pos = st["positions"].long() if st["positions"] is not None else slot
    ang = pos.double()[:, None] * st["freqs"][None, :]
    cos = (ang.cos() * st["scale"]).float()[:, None, :]
    sin = (ang.sin() * st["scale"]).float()[:, None, :]

    def rotate(x):
        y = x.float()
        r = y.clone()
        if c["inter"]:
            a, b = y[..., 0:rot:2], y[..., 1:rot:2]
            r[..., 0:rot:2], r[..., 1:rot:2] = a * cos - b * sin, b * cos + a * sin
        else:
            a, b = y[..., :rot // 2], y[..., rot // 2:rot]
            r[..., :rot // 2], r[..., rot // 2:rot] = a * cos - b * sin, b * cos + a * sin
        return r.to(dt)

    q_out, k_rot = rotate(q), rotate(k)
    page = st["table"].long()[seq, slot // ps]
    st["k_pages"][page, :, slot % ps] = k_rot
    st["v_pages"][page, :, slot % ps] = v
    if st["bounds"] is None:
        return q_out, st["k_pages"], st["v_pages"]
    # bounds of every page that received rows: over its rows held so far
    n_pages = st["n_pages"]
    fill = torch.zeros(n_pages, dtype=torch.long, device=dev)
    fill.scatter_reduce_(0, page, slot % ps + 1, "amax")
    row = torch.arange(ps, device=dev)
    held = (row[None, :] < fill[:, None])[:, None, :, None]
    kf = st["k_pages"].float()
    lo = torch.where(held, kf, torch.full_like(kf, math.inf)).amin(2).to(dt)
    hi = torch.where(held, kf, torch.full_like(kf, -math.inf)).amax(2).to(dt)
    # rows in front of the first new one were held before: their old bound counts as it was
    first = torch.full((n_pages,), ps, dtype=torch.long, device=dev)
    first.scatter_reduce_(0, page, slot % ps, "amin")
    new = ((row[None, :] >= first[:, None]) & (row[None, :] < fill[:, None]))[:, None, :, None]
    nlo = torch.where(new, kf, torch.full_like(kf, math.inf)).amin(2).to(dt)
    nhi = torch.where(new, kf, torch.full_like(kf, -math.inf)).amax(2).to(dt)
    kmin, kmax = st["bounds"]
    touched = (fill > 0)[:, None, None]
    part = touched & (first > 0)[:, None, None]
    kmin.copy_(torch.where(part, torch.minimum(kmin, nlo), torch.where(touched, lo, kmin)))
    kmax.copy_(torch.where(part, torch.maximum(kmax, nhi), torch.where(touched, hi, kmax)))
    return q_out, st["k_pages"], st["v_pages"], kmin, kmax


def _rows(pages_tensor, ids, count):
    """Rows [Hkv, count, d] in fp32 of the pages `ids`, in order."""
    x = pages_tensor[ids].float()                       # [P, Hkv, ps, d]
    x = x.permute(1, 0, 2, 3).reshape(x.shape[1], -1, x.shape[3])
    return x[:, :count]


def _plain_attend(st):
    c = st["case"]
    Hq, Hkv, d, ps = c["Hq"], c["Hkv"], c["d"], c["page"]
    G = Hq // Hkv
    o = torch.zeros((st["n"], Hq, d), dtype=DT[c["dtype"]], device="cuda")
    lse = torch.full((st["n"], Hq), -math.inf, dtype=torch.float32, device="cuda")
    for s, (ql, kl) in enumerate(zip(st["ql"], st["kl"])):
        if ql == 0 or kl == 0:
            continue
        ids = st["table"][s, :(kl + ps - 1) // ps].long()
        K, V = _rows(st["k_pages"], ids, kl), _rows(st["v_pages"], ids, kl)
        key = torch.arange(kl, device="cuda")
        step = max(1, (1 << 28) // (Hq * kl))           # query rows a piece: ~1 GB of scores
        for a in range(0, ql, step):
            b = min(ql, a + step)
            t0 = st["cu"][s] + a
            qf = st["q"][t0:t0 + b - a].float().view(b - a, Hkv, G, d).permute(1, 0, 2, 3)
            x = torch.matmul(qf.reshape(Hkv, -1, d), K.transpose(1, 2)) * (1.0 / math.sqrt(d))
            last = torch.arange(kl - ql + a, kl - ql + b, device="cuda").repeat_interleave(G)
            x.masked_fill_(key[None, None, :] > last[None, :, None], -math.inf)
            m = x.amax(2, keepdim=True)
            x = x.sub_(m).exp_()
            z = x.sum(2, keepdim=True)
            y = torch.matmul(x, V) / z
            o[t0:t0 + b - a] = y.view(Hkv, b - a, G, d).permute(1, 0, 2, 3).reshape(b - a, Hq, d)
            l = (m + z.log()).view(Hkv, b - a, G).permute(1, 0, 2)
            lse[t0:t0 + b - a] = l.reshape(b - a, Hq)
    return o, lse


def _plain_select(st):
    c = st["case"]
    Hq, Hkv, d, ps = c["Hq"], c["Hkv"], c["d"], c["page"]
    S, K, R = c["n_sink"], c["n_top"], c["n_recent"]
    N = S + K + R
    kmin, kmax = st["bounds"]
    pages = torch.full((st["n"], Hkv, N), -1, dtype=torch.int32, device="cuda")
    counts = torch.zeros((st["n"], Hkv), dtype=torch.int32, device="cuda")
    for s, (ql, kl) in enumerate(zip(st["ql"], st["kl"])):
        ids = st["table"][s, :(kl + ps - 1) // ps].long()
        # scores decide which whole numbers come out, so they are formed in 64 bits and rounded once
        mn, mx = kmin[ids].double(), kmax[ids].double()             # [P, Hkv, d]
        for i in range(ql):
            t = st["cu"][s] + i
            vis = (kl - ql + i) // ps + 1
            m = min(vis, N)
            counts[t] = m
            if vis <= N:
                pages[t, :, :m] = torch.arange(vis, device="cuda", dtype=torch.int32)
                continue
            qd = st["q"][t].double().view(Hkv, Hq // Hkv, d)
            up = qd.clamp(min=0).sum(1)
            dn = qd.clamp(max=0).sum(1)
            score = ((up * mx[:vis]).sum(2) + (dn * mn[:vis]).sum(2)).float().t()   # [Hkv, vis]
            mid = score[:, S:vis - R]
            best = torch.sort(mid, dim=1, descending=True, stable=True).indices[:, :K]
            best = best.sort(dim=1).values + S
            pages[t, :, :S] = torch.arange(S, device="cuda", dtype=torch.int32)
            pages[t, :, S:S + K] = best.int()
            pages[t, :, S + K:] = torch.arange(vis - R, vis, device="cuda", dtype=torch.int32)
    return pages, counts


def _plain_selected(st, pages, counts):
    c = st["case"]
    Hq, Hkv, d, ps = c["Hq"], c["Hkv"], c["d"], c["page"]
    G = Hq // Hkv
    N = pages.shape[2]
    o = torch.empty((st["n"], Hq, d), dtype=DT[c["dtype"]], device="cuda")
    lse = torch.empty((st["n"], Hq), dtype=torch.float32, device="cuda")
    head = torch.arange(Hkv, device="cuda")[:, None]
    row = torch.arange(ps, device="cuda")
    for s, (ql, kl) in enumerate(zip(st["ql"], st["kl"])):
        for i in range(ql):
            t = st["cu"][s] + i
            logical = pages[t].long()                                # [Hkv, N]
            live = torch.arange(N, device="cuda")[None, :] < counts[t].long()[:, None]
            logical = torch.where(live, logical, torch.zeros_like(logical))
            ids = st["table"][s].long()[logical]
            K = st["k_pages"][ids, head].float().reshape(Hkv, N * ps, d)
            V = st["v_pages"][ids, head].float().reshape(Hkv, N * ps, d)
            key = (logical[:, :, None] * ps + row).reshape(Hkv, N * ps)
            see = (key <= kl - ql + i) & live[:, :, None].expand(-1, -1, ps).reshape(Hkv, N * ps)
            x = torch.matmul(st["q"][t].float().view(Hkv, G, d), K.transpose(1, 2)) / math.sqrt(d)
            x = x.masked_fill(~see[:, None, :], -math.inf)
            m = x.amax(2, keepdim=True)
            x = (x - m).exp()
            z = x.sum(2, keepdim=True)
            o[t] = (torch.matmul(x, V) / z).reshape(Hq, d)
            lse[t] = (m + z.log()).reshape(Hq)
    return o, lse


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    Hq, Hkv, d, ps = case["Hq"], case["Hkv"], case["d"], case["page"]
    G = Hq // Hkv
    ql, kl = _lengths(case)
    n = sum(ql)
    op = case["op"]
    if op == "append":
        b = 2 * n * (Hq + 2 * Hkv) * d * 2
        if case["bounds"]:
            touched = sum((k - 1) // ps - (k - q) // ps + 1 for q, k in zip(ql, kl) if q)
            b += touched * 2 * Hkv * d * 2
        return {"bytes": b, "flops": 3 * n * (Hq + Hkv) * case["rot"]}
    io = n * Hq * (2 * d * 2 + 4)                  # q read, o and lse written
    if op == "attend":
        pairs = sum(q * (k - q) + q * (q + 1) // 2 for q, k in zip(ql, kl))
        rows = sum(k for q, k in zip(ql, kl) if q)
        return {"bytes": io + rows * Hkv * d * 2 * 2, "flops": 4 * d * Hq * pairs}
    N = case["n_top"] + case["n_sink"] + case["n_recent"]
    by = fl = 0
    for q, k in zip(ql, kl):
        vis = (k - 1) // ps + 1
        if op in ("select", "sparse"):
            if vis > N:
                by += vis * Hkv * 2 * d * 2
                fl += q * vis * Hkv * 2 * d * 2
            by += q * Hkv * (min(vis, N) + 1) * 4 + (q * Hq * d * 2 if op == "select" else 0)
        if op in ("selected", "sparse"):
            rows = min(k, N * ps)
            by += rows * Hkv * d * 2 * 2
            fl += 4 * d * G * Hkv * rows * q
    return {"bytes": by + (io if op != "select" else 0), "flops": fl}


# ------------------------------------------------------------------ the definition in 64 bits
def exact(case, seed):
    """What `run` returns, from the definitions alone; None where that takes long."""
    if work(case)["flops"] > 4e12:
        return None
    st = prepare(case, seed)
    op = case["op"]
    if op == "append":
        return _exact_append(st)
    if op == "select":
        return _exact_pages(st)
    if op == "attend":
        return _exact_attention(st, None, None)
    if op == "selected":
        return _exact_attention(st, st["pages"].tolist(), st["counts"].tolist())
    pages, counts = _exact_pages(st)
    return (pages, counts) + _exact_attention(st, pages.tolist(), counts.tolist())


def _token_places(st):
    """(sequence, slot) of every token, on the host."""
    return [(s, kl - ql + i) for s, (ql, kl) in enumerate(zip(st["ql"], st["kl"]))
            for i in range(ql)]


def _exact_append(st):
    c = st["case"]
    rot, ps, Hq, Hkv, d = c["rot"], c["page"], c["Hq"], c["Hkv"], c["d"]
    places = _token_places(st)
    pos = [p for _, p in places] if st["positions"] is None else st["positions"].tolist()
    x = st["qkv"].double().view(st["n"], Hq + 2 * Hkv, d)
    # complex form: a rotated pair is one number times scale * exp(i angle)
    turn = torch.polar(torch.full((st["n"], rot // 2), float(st["scale"]), dtype=torch.float64,
                                  device="cuda"),
                       torch.tensor(pos, dtype=torch.float64, device="cuda")[:, None]
                       * st["freqs"][None])
    xr = x[:, :Hq + Hkv].clone()
    first, second = ((slice(0, rot, 2), slice(1, rot, 2)) if c["inter"]
                     else (slice(0, rot // 2), slice(rot // 2, rot)))
    z = torch.complex(xr[..., first].contiguous(), xr[..., second].contiguous()) * turn[:, None, :]
    xr[..., first], xr[..., second] = z.real, z.imag
    table = st["table"].tolist()
    page = torch.tensor([table[s][p // ps] for s, p in places], device="cuda")
    row = torch.tensor([p % ps for _, p in places], device="cuda")
    kp, vp = st["k_pages"].double(), st["v_pages"].double()
    kp[page, :, row] = xr[:, Hq:]
    vp[page, :, row] = x[:, Hq + Hkv:]
    out = (xr[:, :Hq], kp, vp)
    if st["bounds"] is None:
        return out
    lo, hi = (b.double().clone() for b in st["bounds"])
    at = 0
    for s, (ql, kl) in enumerate(zip(st["ql"], st["kl"])):
        a = kl - ql
        for pg in range(a // ps, (kl - 1) // ps + 1 if ql else a // ps):
            r0, r1 = max(a, pg * ps), min(kl, (pg + 1) * ps)
            keys = xr[at + r0 - a:at + r1 - a, Hq:]
            new_lo, new_hi = keys.amin(0), keys.amax(0)
            phys = table[s][pg]
            if r0 > pg * ps:
                new_lo = torch.minimum(new_lo, lo[phys])
                new_hi = torch.maximum(new_hi, hi[phys])
            lo[phys], hi[phys] = new_lo, new_hi
        at += ql
    return out + (lo, hi)


def _exact_pages(st):
    c = st["case"]
    ps, S, K, R, Hkv = c["page"], c["n_sink"], c["n_top"], c["n_recent"], c["Hkv"]
    pages = np.full((st["n"], Hkv, S + K + R), -1, dtype=np.int32)
    counts = np.zeros((st["n"], Hkv), dtype=np.int32)
    table = st["table"].tolist()
    for t, (s, p) in enumerate(_token_places(st)):
        vis = p // ps + 1
        if vis <= S + K + R:
            pages[t, :, :vis] = np.arange(vis)
            counts[t] = vis
            continue
        ids = torch.tensor(table[s][:vis], device="cuda")
        lo, hi = st["bounds"][0][ids].double(), st["bounds"][1][ids].double()
        total = torch.zeros((vis, Hkv), dtype=torch.float64, device="cuda")
        G = c["Hq"] // Hkv
        for gq in range(G):
            q = st["q"][t].double().view(Hkv, G, c["d"])[:, gq]
            total += torch.maximum(q * lo, q * hi).sum(2)
        sc = total.float().cpu().numpy()
        for h in range(Hkv):
            mid = sorted(range(S, vis - R), key=lambda j: (-sc[j, h], j))[:K]
            pages[t, h] = list(range(S)) + sorted(mid) + list(range(vis - R, vis))
        counts[t] = S + K + R
    return torch.from_numpy(pages).cuda(), torch.from_numpy(counts).cuda()


def _exact_attention(st, pages, counts):
    c = st["case"]
    Hq, Hkv, d, ps = c["Hq"], c["Hkv"], c["d"], c["page"]
    G = Hq // Hkv
    o = torch.zeros((st["n"], Hq, d), dtype=torch.float64, device="cuda")
    lse = torch.full((st["n"], Hq), -math.inf, dtype=torch.float64, device="cuda")
    for s, (ql, kl) in enumerate(zip(st["ql"], st["kl"])):
        if not ql:
            continue
        for h in range(Hkv):
            ids = st["table"][s, :(kl + ps - 1) // ps].long()
            K = st["k_pages"][ids, h].reshape(-1, d)[:kl].double()
            V = st["v_pages"][ids, h].reshape(-1, d)[:kl].double()
            piece = ql if pages is None else 1
            piece = max(1, min(piece, (1 << 26) // kl // G))
            for a in range(0, ql, piece):
                b = min(ql, a + piece)
                t = st["cu"][s] + a
                q = st["q"][t:t + b - a, h * G:(h + 1) * G].double().reshape(-1, d)
                w = q @ K.t() / math.sqrt(d)
                at = torch.arange(kl, device="cuda")
                lim = (kl - ql + a) + torch.arange(b - a, device="cuda").repeat_interleave(G)
                seen = at[None, :] <= lim[:, None]
                if pages is not None:
                    chosen = torch.zeros(ids.numel(), dtype=torch.bool, device="cuda")
                    chosen[torch.tensor(pages[t][h][:counts[t][h]], device="cuda",
                                        dtype=torch.long)] = True
                    seen = seen & chosen.repeat_interleave(ps)[:kl][None, :]
                w = torch.where(seen, w, torch.full_like(w, -math.inf))
                z = torch.logsumexp(w, 1)
                w = torch.exp(w - z[:, None])
                o[t:t + b - a, h * G:(h + 1) * G] = (w @ V).view(b - a, G, d)
                lse[t:t + b - a, h * G:(h + 1) * G] = z.view(b - a, G)
    return o, lse
