"""Measured cases of a batch of draft trees over the paged cache.

Four operators make one step of several streams that each verify a draft tree:
attention of the trees' nodes over the pages, the logits of the nodes under
repetition penalties, biases and grammar masks, the move of the accepted rows
to the end of the cache in every layer, and the token counts that the
penalties read.  Each case holds plain numbers; `run` makes one pass, in
elementary torch operations or (`own`) through the library's calls; `exact` is
the definition in 64 bits.
"""
import math
import random

import torch

own = False

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
MOST_ATTEND = 4.0e11        # operations of the largest listed tree case
MOST_LOGITS = 1024 * 128256


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # trees of a few nodes on three short streams, tiny layer: latency only
        dict(name="tree_tiny", op="tree", n_seq=3, q=5, kv=4096, Hq=4, Hkv=1, d=64, page=16,
             dtype="bf16", ragged=True, shape=1),
        # one stream verifying 64 nodes at 100K tokens, 8B-shaped layer
        dict(name="tree_100k", op="tree", n_seq=1, q=64, kv=102400, Hq=32, Hkv=8, d=128, page=64,
             dtype="bf16", ragged=False, shape=2),
        # short streams with trees of 1 to 64 nodes in one call, small heads
        dict(name="tree_mixed", op="tree", n_seq=9, q=64, kv=6000, Hq=16, Hkv=4, d=64, page=32,
             dtype="fp16", ragged=True, shape=3),
        # twelve streams verifying full trees, 14B-shaped layer: the largest
        dict(name="tree_batch", op="tree", n_seq=12, q=64, kv=24576, Hq=40, Hkv=8, d=128, page=32,
             dtype="fp16", ragged=False, shape=4),
        # accepted rows of one stream, 1.5B-shaped model: latency only
        dict(name="commit_one", op="commit", layers=28, n_seq=1, q=64, kv=102400, Hkv=2, d=128,
             page=16, dtype="bf16", bounds=False, ragged=False, shape=5),
        # accepted rows of sixteen streams with the pages' key bounds, 8B-shaped model
        dict(name="commit_batch", op="commit", layers=32, n_seq=16, q=64, kv=32768, Hkv=8, d=128,
             page=32, dtype="bf16", bounds=True, ragged=True, shape=6),
        # the tokens that a step of sixteen streams accepted
        dict(name="counts_step", op="counts", n_seq=16, tokens=8, V=128256, reset=False,
             prompt=False, ragged=True, shape=7),
        # eight streams taken up again with up to 100K generated tokens
        dict(name="counts_resume", op="counts", n_seq=8, tokens=102400, V=151936, reset=True,
             prompt=False, ragged=True, shape=8),
        # next token of four streams with a repetition penalty: latency only
        dict(name="logits_decode", op="logits", n_seq=4, q=1, V=32000, pad=0, dtype="bf16",
             history=2000, counts=False, tree=False, bias=0, masks="none", ragged=False, shape=9),
        # 64 nodes of one stream, every penalty, rows of a padded output layer
        dict(name="logits_tree", op="logits", n_seq=1, q=64, V=151936, pad=128, dtype="fp32",
             history=100000, counts=True, tree=True, bias=0, masks="none", ragged=False,
             shape=10),
        # next token of a ragged batch, odd vocabulary, biases and a few shared masks
        dict(name="logits_odd", op="logits", n_seq=48, q=1, V=32003, pad=0, dtype="fp16",
             history=5000, counts=True, tree=False, bias=300, masks="shared", ragged=False,
             shape=11),
        # sixteen streams with full trees under a grammar, a mask a node
        dict(name="logits_grammar", op="logits", n_seq=16, q=64, V=128256, pad=0, dtype="bf16",
             history=20000, counts=True, tree=True, bias=64, masks="each", ragged=False,
             shape=12),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["tree", "tree", "tree", "commit", "counts", "logits", "logits"])
    c = dict(op=op, n_seq=log(1, 16), ragged=rng.random() < 0.6, shape=rng.randrange(1 << 30))
    if op in ("tree", "commit"):
        Hq, Hkv = rng.choice([(4, 1), (12, 2), (16, 4), (32, 8), (40, 8), (8, 8)])
        c.update(Hkv=Hkv, q=log(1, 64), d=rng.choice([64, 128, 128]),
                 page=rng.choice([16, 32, 64, 128]), dtype=rng.choice(["bf16", "fp16"]))
    if op == "tree":
        top = min(102400, 300000 // c["n_seq"],
                  int(MOST_ATTEND / (4.0 * c["n_seq"] * c["q"] * Hq * c["d"])))
        c.update(Hq=Hq, kv=log(c["q"], max(c["q"], top)))
    elif op == "commit":
        c.update(layers=log(1, 32), kv=log(c["q"], 102400), bounds=rng.random() < 0.5)
    elif op == "counts":
        reset = rng.random() < 0.5
        c.update(tokens=log(1, 102400 if reset else 64), V=log(1000, 152064), reset=reset,
                 prompt=rng.random() < 0.3)
    else:
        tree = rng.random() < 0.5
        V = log(1000, 152064)
        n_seq = log(1, 64)
        c.update(n_seq=n_seq, q=log(1, max(1, min(64, MOST_LOGITS // (V * n_seq)))) if tree else 1,
                 V=V, pad=rng.choice([0, 0, 0, 5, 64]), dtype=rng.choice(["bf16", "fp16", "fp32"]),
                 history=log(1, 102400 // n_seq), counts=rng.random() < 0.6, tree=tree,
                 bias=rng.choice([0, 0, log(1, 300)]),
                 masks=rng.choice(["none", "shared", "each"]))
    return c


def _lengths(case):
    """New tokens and rows (new ones included) of every sequence."""
    rng = random.Random(case["shape"])
    n, q = case["n_seq"], case["q"]
    kv = case.get("kv", q)
    if not case["ragged"]:
        return [q] * n, [max(kv, q)] * n
    ql = [q if q == 1 else rng.choice([q, rng.randint(1, q), rng.randint(1, q)]) for _ in range(n)]
    kl = [max(ql[i], rng.randint(max(1, kv // 8), kv)) for i in range(n)]
    kl[-1] = max(kv, ql[-1])
    if n > 2 and q > 1:
        ql[0] = 0 if case["op"] == "tree" else ql[0]       # a stream with nothing new in this call
        ql[1] = 1                                          # and one that drafted nothing
    return ql, kl


def _token_lengths(case):
    rng = random.Random(case["shape"])
    m = case["tokens"]
    if not case["ragged"]:
        return [m] * case["n_seq"]
    return [rng.randint(0, m) for _ in range(case["n_seq"] - 1)] + [m]


# ------------------------------------------------------------------ inputs
def _trees(host, ql):
    """Parents of every tree's nodes, packed: three children a node, or any earlier node."""
    out = []
    for n in ql:
        out += [-1 if i == 0 else (i - 1) // 3 if host.random() < 0.6 else host.randrange(i)
                for i in range(n)]
    return out


def _cu(ql):
    cu = [0]
    for x in ql:
        cu.append(cu[-1] + x)
    return cu


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    host = random.Random(seed)

    def ints(x):
        return torch.tensor(x, dtype=torch.int32, device="cuda")

    if case["op"] == "counts":
        return _prepare_counts(case, g, ints)
    ql, kl = _lengths(case)
    cu = _cu(ql)
    st = dict(case=case, ql=ql, kl=kl, cu=cu, n=cu[-1], cu_q=ints(cu), seq_lens=ints(kl))
    parents = _trees(host, ql)
    st["parents"] = ints(parents)
    if case["op"] == "logits":
        return _prepare_logits(case, st, g, host, ints)
    dt, Hkv, d, ps = DT[case["dtype"]], case["Hkv"], case["d"], case["page"]

    def normal(*shape):
        return torch.empty(shape, dtype=dt, device="cuda").normal_(generator=g)

    pages_of = [(x + ps - 1) // ps for x in kl]
    if case["op"] == "tree":
        first = [0] * len(kl)
    else:
        # the streams share their pages up to the trees' (one prompt): the move reads none of them
        first = [max(0, (k - q) // ps) for q, k in zip(ql, kl)]
    n_pages = 1 + sum(p - f for p, f in zip(pages_of, first)) + 2
    perm = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    table = perm[0].repeat(len(kl), max(pages_of))
    at = 1
    for s, (p, f) in enumerate(zip(pages_of, first)):
        table[s, f:p] = perm[at:at + p - f]
        at += p - f
    st.update(table=table, n_pages=n_pages)
    if case["op"] == "tree":
        st["q"] = normal(st["n"], case["Hq"], d)
        st["k_pages"] = normal(n_pages, Hkv, ps, d)
        st["v_pages"] = normal(n_pages, Hkv, ps, d)
        # heavy hitters: one row of every fortieth page points along the last node's queries
        for s in range(len(ql)):
            if ql[s]:
                hot = table[s, :pages_of[s]][host.randrange(0, 3)::40].long()
                dirn = st["q"][cu[s + 1] - 1].view(Hkv, -1, d).float().mean(1)
                row = host.randrange(ps)
                st["k_pages"][hot, :, row] = (st["k_pages"][hot, :, row].float()
                                              + 1.5 * dirn).to(dt)
        return st
    # the accepted path: from a root to one of its nodes
    path = torch.full((len(ql), case["q"]), -2, dtype=torch.int32)
    n_path = []
    for s in range(len(ql)):
        a, nodes = host.randrange(ql[s]), []
        while a >= 0:
            nodes.append(a)
            a = parents[cu[s] + a]
        path[s, :len(nodes)] = torch.tensor(nodes[::-1], dtype=torch.int32)
        n_path.append(len(nodes))
    st["path"], st["n_path"] = path.cuda(), ints(n_path)
    ly = case["layers"]
    st["k_pages"] = normal(ly, n_pages, Hkv, ps, d)
    st["v_pages"] = normal(ly, n_pages, Hkv, ps, d)
    st["layers"] = _addresses(st["k_pages"], st["v_pages"])
    st["bounds"] = None
    if case["bounds"]:
        st["bounds"] = (st["k_pages"].amin(3).contiguous(), st["k_pages"].amax(3).contiguous())
        st["bound_layers"] = _addresses(*st["bounds"])
    return st


def _addresses(a, b):
    """Where each layer's part of two stacked tensors lies, for a call over all layers."""
    host = [[x.data_ptr() + i * x.stride(0) * x.element_size() for i in range(x.shape[0])]
            for x in (a, b)]
    return torch.tensor(host, dtype=torch.int64).cuda()


def _zipf(g, shape, V):
    """Token ids, the small ones often."""
    u = torch.rand(shape, generator=g, device="cuda", dtype=torch.float64)
    return (u.pow(4.0) * V).long().clamp_(max=V - 1).to(torch.int32)


def _prepare_counts(case, g, ints):
    lens, V, n = _token_lengths(case), case["V"], case["n_seq"]
    st = dict(case=case, lens=lens, tokens=_zipf(g, (n, case["tokens"]), V), n_new=ints(lens))
    # what the streams have generated before
    old = _zipf(g, (n, 3000), V)
    st["counts"], st["seen"] = _count(old, torch.ones_like(old, dtype=torch.bool), V)
    return st


def _prepare_logits(case, st, g, host, ints):
    n, V, ns = st["n"], case["V"], case["n_seq"]
    full = torch.empty((n, V + case["pad"]), device="cuda").normal_(generator=g).mul_(2.5)
    st["logits"] = full.to(DT[case["dtype"]])[:, :V]
    old = _zipf(g, (ns, case["history"]), V)
    st["counts"], st["seen"] = _count(old, torch.ones_like(old, dtype=torch.bool), V)
    if not case["counts"]:
        st["counts"] = None

    def each(lo, hi):
        return torch.tensor([host.uniform(lo, hi) for _ in range(ns)], device="cuda")

    st["repetition"] = each(1.0, 1.4)
    st["frequency"] = each(0.0, 0.5) if case["counts"] else None
    st["presence"] = each(0.0, 0.8) if case["counts"] else None
    st["tokens"] = _zipf(g, (n,), V) if case["tree"] else None
    if not case["tree"]:
        st["parents"] = None
    st["bias_ids"] = st["bias"] = None
    if case["bias"]:
        m = min(case["bias"], V)
        ids = torch.rand((ns, V), generator=g, device="cuda").argsort(1)[:, :m].to(torch.int32)
        st["bias_ids"] = ids.contiguous()
        st["bias"] = torch.empty((ns, m), device="cuda").normal_(generator=g).mul_(5.0)
    st["mask"] = st["mask_rows"] = None
    if case["masks"] != "none":
        rows = n if case["masks"] == "each" else 4
        # one in eight tokens allowed, as where a grammar expects a number or a key
        words = (V + 31) // 32
        a = torch.randint(-2 ** 31, 2 ** 31, (3, rows, words), generator=g, device="cuda")
        st["mask"] = (a[0] & a[1] & a[2]).to(torch.int32)
        if case["masks"] == "shared":       # some rows are free
            st["mask_rows"] = ints([host.randrange(-1, 4) for _ in range(n)])
    return st


# ------------------------------------------------------------------ one pass
def run(state):
    if own:
        return _run_own(state)
    op = state["case"]["op"]
    if op == "tree":
        return _plain_tree(state)
    if op == "commit":
        return _plain_commit(state)
    if op == "counts":
        return _plain_counts(state)
    return _plain_logits(state)


def _run_own(st):
    import self_speculative_ultra_gb300 as ts
    c = st["case"]
    if c["op"] == "tree":
        return ts.ts_paged_tree_attention(st["q"], st["k_pages"], st["v_pages"], st["cu_q"],
                                          st["seq_lens"], st["table"], st["parents"],
                                          max_q=max(st["ql"]))
    if c["op"] == "commit":
        more = {}
        if st["bounds"]:
            more = dict(key_min=st["bounds"][0], key_max=st["bounds"][1],
                        bounds_table=st["bound_layers"])
        new = ts.ts_paged_kv_commit(st["k_pages"], st["v_pages"], st["cu_q"], st["seq_lens"],
                                    st["table"], st["path"], st["n_path"], table=st["layers"],
                                    **more)
        out = (new, st["k_pages"], st["v_pages"])
        return out + tuple(st["bounds"]) if st["bounds"] else out
    if c["op"] == "counts":
        ts.ts_token_counts(st["tokens"], st["n_new"], c["V"], st["seen"], counts=st["counts"],
                           reset=c["reset"], prompt=c["prompt"])
        return st["counts"], st["seen"]
    return ts.ts_logits_process(st["logits"], st["cu_q"], seen=st["seen"], counts=st["counts"],
                                repetition=st["repetition"], frequency=st["frequency"],
                                presence=st["presence"], tree_tokens=st["tokens"],
                                parents=st["parents"], bias_ids=st["bias_ids"], bias=st["bias"],
                                mask=st["mask"], mask_rows=st["mask_rows"])


def _pad(st, T):
    """(token of each node [n_seq, T], which nodes there are) of the packed batch."""
    cu = st["cu_q"].long()
    i = torch.arange(T, device="cuda")
    live = i[None, :] < (cu[1:] - cu[:-1])[:, None]
    return (cu[:-1, None] + i).clamp(max=max(st["n"] - 1, 0)), live


def _ancestors(st, T, tok, live):
    """[n_seq, T, T]: whether column a is row i's node or one of its ancestors."""
    par = st["parents"].long()[tok].masked_fill(~live, -1)
    i = torch.arange(T, device="cuda")
    m = ((par[:, :, None] == i) | (i[:, None] == i)).float()
    m = (m @ m).clamp(max=1.0)          # paths of up to 2, 4, .. 64 edges
    m = (m @ m).clamp(max=1.0)
    m = (m @ m).clamp(max=1.0)
    m = (m @ m).clamp(max=1.0)
    m = (m @ m).clamp(max=1.0)
    m = (m @ m).clamp(max=1.0)
    return (m > 0) & live[:, :, None]


def _plain_tree(st):
    c = st["case"]
    Hq, Hkv, d, T, ns = c["Hq"], c["Hkv"], c["d"], c["q"], c["n_seq"]
    G = Hq // Hkv
    tok, live = _pad(st, T)
    anc = _ancestors(st, T, tok, live)
    kl = st["seq_lens"].long()
    L = kl - live.sum(1)
    ids = st["table"].long()
    KV = ids.shape[1] * c["page"]

    def rows(pages):                    # [n_seq, Hkv, KV, d] in 32 bits
        return pages[ids].permute(0, 2, 1, 3, 4).reshape(ns, Hkv, KV, d).float()

    q = st["q"].float()[tok].view(ns, T, Hkv, G, d).permute(0, 2, 1, 3, 4).reshape(ns, Hkv, -1, d)
    x = torch.matmul(q, rows(st["k_pages"]).transpose(2, 3)) * (1.0 / math.sqrt(d))
    at = torch.arange(KV, device="cuda")[None, :] - L[:, None]
    see = anc.gather(2, at.clamp(0, T - 1)[:, None, :].expand(-1, T, -1))
    see = (see & (at < T)[:, None, :]) | (at < 0)[:, None, :]
    x = x.view(ns, Hkv, T, G, KV).masked_fill_(~see[:, None, :, None, :], -math.inf)
    m = x.amax(4, keepdim=True)
    x = x.sub_(m).exp_()
    z = x.sum(4, keepdim=True)
    y = torch.matmul(x.view(ns, Hkv, T * G, KV), rows(st["v_pages"])).view(ns, Hkv, T, G, d) / z
    o = y.permute(0, 2, 1, 3, 4).reshape(ns, T, Hq, d)[live].to(DT[c["dtype"]])
    lse = (m + z.log()).squeeze(4).permute(0, 2, 1, 3).reshape(ns, T, Hq)[live]
    return o, lse


def _plain_commit(st):
    c = st["case"]
    ps, T = c["page"], c["q"]
    cu = st["cu_q"].long()
    kl = st["seq_lens"].long()
    L = kl - (cu[1:] - cu[:-1])
    n_path = st["n_path"].long()
    t = torch.arange(T, device="cuda")
    seq, t = torch.nonzero((t[None, :] >= 1) & (t[None, :] < n_path[:, None]), as_tuple=True)
    src, dst = L[seq] + st["path"].long()[seq, t], L[seq] + t
    table = st["table"].long()
    ps_, pd = table[seq, src // ps], table[seq, dst // ps]
    for x in (st["k_pages"], st["v_pages"]):
        x[:, pd, :, dst % ps] = x[:, ps_, :, src % ps]
    new = torch.where(cu[1:] > cu[:-1], L + n_path, kl).to(torch.int32)
    out = (new, st["k_pages"], st["v_pages"])
    if st["bounds"] is None:
        return out
    # pages that hold a committed row of the tree: over these, and over what was there before
    j = (L // ps)[:, None] + torch.arange((T - 1) // ps + 2, device="cuda")
    first = torch.maximum(j * ps, L[:, None])
    last = torch.minimum((j + 1) * ps, (L + n_path)[:, None])
    s, k = torch.nonzero(first < last, as_tuple=True)
    page, r0, r1 = j[s, k], first[s, k], last[s, k]
    phys = table[s, page]
    row = (page * ps)[:, None] + torch.arange(ps, device="cuda")
    held = ((row >= r0[:, None]) & (row < r1[:, None]))[None, :, None, :, None]
    keys = st["k_pages"][:, phys].float()
    lo = keys.masked_fill(~held, math.inf).amin(3).to(DT[c["dtype"]])
    hi = keys.masked_fill(~held, -math.inf).amax(3).to(DT[c["dtype"]])
    over = (page * ps >= L[s])[None, :, None, None]
    kmin, kmax = st["bounds"]
    kmin[:, phys] = torch.where(over, lo, torch.minimum(lo, kmin[:, phys]))
    kmax[:, phys] = torch.where(over, hi, torch.maximum(hi, kmax[:, phys]))
    return out + (kmin, kmax)


def _count(tokens, live, V):
    """(counts [n_seq, V], seen [n_seq, ceil(V / 32)]) of the live tokens, int32."""
    n, words = tokens.shape[0], (V + 31) // 32
    at = tokens.long() + torch.arange(n, device="cuda")[:, None] * (words * 32)
    counts = torch.zeros(n * words * 32, dtype=torch.int32, device="cuda")
    counts.scatter_add_(0, at.reshape(-1), live.reshape(-1).to(torch.int32))
    counts = counts.view(n, words * 32)
    bit = torch.ones(32, dtype=torch.int64, device="cuda") << torch.arange(32, device="cuda")
    seen = ((counts > 0).view(n, words, 32) * bit).sum(2)
    return counts[:, :V].contiguous(), seen.to(torch.int32)


def _plain_counts(st):
    c = st["case"]
    live = torch.arange(c["tokens"], device="cuda")[None, :] < st["n_new"].long()[:, None]
    counts, seen = _count(st["tokens"], live, c["V"])
    if c["prompt"]:
        counts.zero_()
    if c["reset"]:
        st["counts"].copy_(counts)
        st["seen"].copy_(seen)
    else:
        st["counts"].add_(counts)
        st["seen"].bitwise_or_(seen)
    return st["counts"], st["seen"]


def _bits(words, V):
    """[rows, V] truth values of rows of packed words."""
    b = (words[:, :, None] >> torch.arange(32, dtype=torch.int32, device="cuda")) & 1
    return b.view(words.shape[0], -1)[:, :V] > 0


def _plain_logits(st):
    c = st["case"]
    V, T, n = c["V"], c["q"], st["n"]
    cu = st["cu_q"].long()
    seq = torch.repeat_interleave(torch.arange(c["n_seq"], device="cuda"), cu[1:] - cu[:-1],
                                  output_size=n)
    x = st["logits"].float()
    if st["bias"] is not None:
        add = torch.zeros((c["n_seq"], V), device="cuda")
        add.scatter_(1, st["bias_ids"].long(), st["bias"])
        x = x + add[seq]
    seen = _bits(st["seen"], V)[seq]
    count = st["counts"][seq] if st["counts"] is not None else None
    if st["tokens"] is not None:
        # the drafted tokens on each node's path (the root is in the history already)
        tok, live = _pad(st, T)
        anc = _ancestors(st, T, tok, live) & (torch.arange(T, device="cuda") > 0)
        ids = st["tokens"].long()[tok][seq]
        path = torch.zeros((n, V), dtype=torch.int32, device="cuda")
        path.scatter_add_(1, ids, anc[live].to(torch.int32))
        seen = seen | (path > 0)
        count = count + path if count is not None else None
    rep = st["repetition"][seq][:, None]
    x = torch.where(seen, torch.where(x > 0, x / rep, x * rep), x)
    if count is not None:
        x = x - st["frequency"][seq][:, None] * count.float()
        x = x - st["presence"][seq][:, None] * (count > 0).float()
    if st["mask"] is not None:
        allowed = _bits(st["mask"], V)
        if st["mask_rows"] is not None:
            r = st["mask_rows"].long()
            allowed = allowed[r.clamp(min=0)] | (r < 0)[:, None]
        x = x.masked_fill(~allowed, -math.inf)
    return x


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    op = case["op"]
    if op == "counts":
        lens, V, n = _token_lengths(case), case["V"], case["n_seq"]
        if case["reset"]:
            return {"bytes": 4 * sum(lens) + n * (4 * V + 4 * ((V + 31) // 32)), "flops": sum(lens)}
        return {"bytes": max(20 * sum(lens), 4), "flops": sum(lens)}
    ql, kl = _lengths(case)
    n = sum(ql)
    if op == "tree":
        Hq, Hkv, d = case["Hq"], case["Hkv"], case["d"]
        rows = sum(k for q, k in zip(ql, kl) if q)
        pairs = sum(q * (k - q) + q * min(q, 4) for q, k in zip(ql, kl))
        return {"bytes": n * Hq * (4 * d + 4) + rows * Hkv * d * 4, "flops": 4 * d * Hq * pairs}
    if op == "commit":
        # three moved rows a tree at most on average, K and V read and written
        rows = sum(min(q - 1, 3) for q in ql) * case["layers"] * case["Hkv"]
        b = rows * case["d"] * 2 * 4
        if case["bounds"]:
            b += len(ql) * case["layers"] * case["Hkv"] * case["d"] * 2 * 4
        return {"bytes": max(b, 4 * len(ql)), "flops": rows}
    V, words = case["V"], (case["V"] + 31) // 32
    b = n * V * (4 + (4 if case["dtype"] == "fp32" else 2)) + case["n_seq"] * words * 4
    if case["masks"] != "none":
        b += 4 * words * (n if case["masks"] == "each" else 4)
    return {"bytes": b, "flops": 3 * n * V}


# ------------------------------------------------------------------ the definition in 64 bits
def exact(case, seed):
    """What `run` returns, from the definitions alone, sequence by sequence and node by node."""
    st = prepare(case, seed)
    return {"tree": _exact_tree, "commit": _exact_commit, "counts": _exact_counts,
            "logits": _exact_logits}[case["op"]](st)


def _paths(st):
    """Of every node, packed: its ancestors and itself, root first."""
    par = st["parents"].tolist()
    out = []
    for s, ql in enumerate(st["ql"]):
        for i in range(ql):
            p = par[st["cu"][s] + i]
            out.append((out[st["cu"][s] + p] if p >= 0 else []) + [i])
    return out


def _exact_tree(st):
    c = st["case"]
    Hq, Hkv, d = c["Hq"], c["Hkv"], c["d"]
    G = Hq // Hkv
    paths = _paths(st)
    o = torch.zeros((st["n"], Hq, d), dtype=torch.float64, device="cuda")
    lse = torch.zeros((st["n"], Hq), dtype=torch.float64, device="cuda")
    for s, (ql, kl) in enumerate(zip(st["ql"], st["kl"])):
        if not ql:
            continue
        t0, L = st["cu"][s], kl - ql
        hidden = torch.ones((ql, kl), dtype=torch.bool)
        hidden[:, :L] = False
        for i in range(ql):
            hidden[i, [L + a for a in paths[t0 + i]]] = False
        hidden = hidden.cuda()
        ids = st["table"][s, :(kl + c["page"] - 1) // c["page"]].long()
        for h in range(Hq):
            K = st["k_pages"][ids, h // G].reshape(-1, d)[:kl].double()
            V = st["v_pages"][ids, h // G].reshape(-1, d)[:kl].double()
            w = st["q"][t0:t0 + ql, h].double() @ K.t() / math.sqrt(d)
            w[hidden] = -math.inf
            z = torch.logsumexp(w, 1)
            lse[t0:t0 + ql, h] = z
            o[t0:t0 + ql, h] = torch.exp(w - z[:, None]) @ V
    return o, lse


def _exact_commit(st):
    c = st["case"]
    ps = c["page"]
    k, v = st["k_pages"].double(), st["v_pages"].double()
    lo, hi = (b.double().clone() for b in st["bounds"]) if st["bounds"] else (None, None)
    table, path, n_path = st["table"].tolist(), st["path"].tolist(), st["n_path"].tolist()
    new = []
    for s, (ql, kl) in enumerate(zip(st["ql"], st["kl"])):
        L = kl - ql

        def place(r):
            return table[s][r // ps], r % ps

        for t in range(1, n_path[s]):
            (a, i), (b, j) = place(L + path[s][t]), place(L + t)
            k[:, b, :, j] = k[:, a, :, i]
            v[:, b, :, j] = v[:, a, :, i]
        new.append(L + n_path[s])
        for p in range(L // ps, (L + n_path[s] - 1) // ps + 1):
            if lo is None:
                continue
            phys = table[s][p]
            held = k[:, phys, :, max(L - p * ps, 0):min(ps, L + n_path[s] - p * ps)]
            a, b = held.amin(2), held.amax(2)
            if p * ps < L:
                a, b = torch.minimum(a, lo[:, phys]), torch.maximum(b, hi[:, phys])
            lo[:, phys], hi[:, phys] = a, b
    out = (torch.tensor(new, dtype=torch.int32, device="cuda"), k, v)
    return out + (lo, hi) if lo is not None else out


def _exact_counts(st):
    c = st["case"]
    V = c["V"]
    counts, seen = st["counts"].clone(), _bits(st["seen"], V)
    for s, m in enumerate(st["lens"]):
        got = torch.bincount(st["tokens"][s, :m].long(), minlength=V).to(torch.int32)
        if c["reset"]:
            counts[s], seen[s] = 0, False
        if not c["prompt"]:
            counts[s] += got
        seen[s] |= got > 0
    words = torch.zeros((c["n_seq"], (V + 31) // 32), dtype=torch.int64, device="cuda")
    for b in range(32):
        x = seen[:, b::32].long()
        words[:, :x.shape[1]] += x << b
    return counts, torch.where(words >= 2 ** 31, words - 2 ** 32, words).to(torch.int32)


def _exact_logits(st):
    c = st["case"]
    V = c["V"]
    paths = _paths(st) if st["tokens"] is not None else None
    y = torch.empty((st["n"], V), dtype=torch.float64, device="cuda")
    bit = torch.arange(V, device="cuda")
    bits = {}

    def unpack(words):
        return ((words.long()[bit // 32] >> (bit % 32)) & 1).bool()

    for s in range(c["n_seq"]):
        old = unpack(st["seen"][s])
        for i in range(st["ql"][s]):
            t = st["cu"][s] + i
            x = st["logits"][t].double()
            if st["bias"] is not None:
                x[st["bias_ids"][s].long()] += st["bias"][s].double()
            met = old.clone()
            times = st["counts"][s].double() if st["counts"] is not None else None
            if paths is not None and i:
                drafted = st["tokens"][[st["cu"][s] + a for a in paths[t][1:]]].long()
                met[drafted] = True
                if times is not None:
                    times = times + torch.bincount(drafted, minlength=V)
            r = st["repetition"][s].double()
            x[met] = torch.maximum(x[met], x[met] * 0) / r + torch.minimum(x[met], x[met] * 0) * r
            if times is not None:
                x -= st["frequency"][s].double() * times
                x -= st["presence"][s].double() * (times > 0)
            if st["mask"] is not None:
                row = t if st["mask_rows"] is None else int(st["mask_rows"][t])
                if row >= 0:
                    if c["masks"] == "each":
                        ok = unpack(st["mask"][row])
                    else:
                        ok = bits.setdefault(row, unpack(st["mask"][row]))
                    x[~ok] = -math.inf
            y[t] = x
    return y
