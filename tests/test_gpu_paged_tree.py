"""GPU parity of the draft trees over a paged cache: attention of their nodes
against the 64-bit oracle, and the move of the accepted rows."""
import numpy as np
import pytest
import torch

from oracle import paged_oracle as po
import paged_util as pu

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16
P_ROUND = {BF: 2.0 ** -8, FP: 2.0 ** -11}      # a weight rounded once, where tiles of rows are


@pytest.fixture(scope="module")
def ts():
    import self_speculative_ultra_gb300 as ts
    ts.build()
    return ts


def status_of(b):
    torch.cuda.synchronize()
    return int(b.status.item())


def tree(kind, n, rng):
    """Parents of n nodes."""
    if kind == "chain":
        return [i - 1 for i in range(n)]
    if kind == "star":
        return [-1, *[0] * (n - 1)][:n]
    if kind == "ternary":
        return [-1 if i == 0 else (i - 1) // 3 for i in range(n)]
    return [-1 if i == 0 else int(rng.integers(0, i)) for i in range(n)]


def parents_of(q_lens, kind="any", seed=0, extra=0):
    rng = np.random.default_rng(seed)
    kinds = ["chain", "star", "ternary", "any"] if kind == "mixed" else [kind]
    out = []
    for s, n in enumerate(q_lens):
        out += tree(kinds[s % len(kinds)], n, rng)
    return torch.tensor(out + [-9] * extra, dtype=torch.int32, device="cuda")


def attend(ts, b, par, **kw):
    o = torch.full((b.n, b.Hq, b.d), 55.0, dtype=b.dtype, device="cuda")
    lse = torch.full((b.n, b.Hq), 55.0, dtype=torch.float32, device="cuda")
    kw.setdefault("max_q", b.max_q)
    ts.ts_paged_tree_attention(b.q, b.k, b.v, b.cu_q, b.lens, b.table, par, o=o, lse=lse,
                               status=b.status, **kw)
    assert status_of(b) == 0
    end = b.cu[-1]
    assert (o[end:] == 55.0).all() and (lse[end:] == 55.0).all()
    return o, lse


def oracle(b, par):
    return po.tree_attention(pu.f64(b.q), pu.f64(b.k), pu.f64(b.v), b.cu, b.kv_lens,
                             b.table_host.numpy(), par.cpu().numpy())


def check(ts, b, par, **kw):
    o, lse = attend(ts, b, par, **kw)
    pu.check_attention(o, lse, oracle(b, par), b.dtype, b.d, p_round=P_ROUND[b.dtype])
    return o, lse


@pytest.mark.parametrize("dtype", [BF, FP], ids=["bf16", "fp16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("ps", [16, 32, 64, 128])
def test_trees(ts, dtype, d, ps):
    """Chains, stars, ternary and random trees, single nodes, streams without a
    node and a tree without a cache, in one call; trees that cross pages and tiles."""
    b = pu.Batch([40, 0, 1, 64, 7, 33, 2], [100, 40, 300, 500, 7, 129, 1030], 4, 2, d, ps, dtype,
                 seed=20 + ps, extra=5)
    check(ts, b, parents_of(b.q_lens, "mixed", seed=ps, extra=5))


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (5, 1), (12, 2), (40, 8), (16, 1), (7, 7)])
@pytest.mark.parametrize("q,kv", [(1, 1), (2, 2), (13, 400), (64, 64), (64, 1111), (31, 4099)])
def test_tree_head_groups(ts, Hq, Hkv, q, kv):
    b = pu.Batch([q, (q + 1) // 2], [kv, kv], Hq, Hkv, 128, 64, BF, seed=Hq + q)
    check(ts, b, parents_of(b.q_lens, "any", seed=q))


@pytest.mark.parametrize("dtype", [BF, FP], ids=["bf16", "fp16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kind", ["chain", "star", "ternary", "any"])
def test_tiles_of_rows(ts, dtype, d, kind):
    """Many rows over long caches: the trees stand at every place of a 128-key tile."""
    lens = [20000, 9001, 9064, 9100, 9215, 9216, 9280]
    b = pu.Batch([64, 64, 64, 64, 63, 64, 50], lens, 16, 2, d, 32, dtype, seed=31)
    check(ts, b, parents_of(b.q_lens, kind, seed=2))


def _streams(n, seed, top, kv):
    """Nodes and lengths of n streams, some without nodes, some without a cache."""
    rng = np.random.default_rng(seed)
    q = [0 if x < 0.2 else int(rng.integers(1, top + 1)) for x in rng.random(n)]
    q[n // 2] = top
    k = [a if x < 0.1 else a + int(rng.integers(0, kv)) for a, x in zip(q, rng.random(n))]
    return q, k


@pytest.mark.parametrize("dtype", [BF, FP], ids=["bf16", "fp16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n,top,kv,Hq,Hkv", [
    (1, 64, 60000, 8, 2),          # one tile a KV head, cut many times
    (1, 64, 30000, 2, 1),          # of one group
    (5, 64, 9000, 12, 3),
    (100, 64, 1500, 4, 2),         # more tiles than SMs
    (40, 32, 4000, 8, 4),
    (700, 33, 300, 4, 1),          # more streams than threads
    (90, 64, 700, 4, 4),
])
def test_lines_of_tiles(ts, dtype, d, n, top, kv, Hq, Hkv):
    """Trees of one tile: stretches over many streams, cut tiles, streams without nodes."""
    q, k = _streams(n, n + top, top, kv)
    if n == 1:
        k = [kv]
    b = pu.Batch(q, k, Hq, Hkv, d, 32, dtype, seed=n, extra=2)
    par = parents_of(q, "mixed", seed=n, extra=2)
    o, lse = check(ts, b, par)
    o2, lse2 = attend(ts, b, par)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    check(ts, b, par, max_kv=64)                   # the host's hint is far too short
    need = ts.ts_paged_tree_attention_workspace_bytes(b.n, n, Hq, Hkv, d, b.table.shape[1], 32, top)
    ws = torch.full((max(need, 1) + 256,), 255, dtype=torch.uint8, device="cuda")
    ws = ws[(-ws.data_ptr()) % 256:][:max(need, 1)]
    o2, lse2 = attend(ts, b, par, workspace=ws)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("last", [0, 64])
@pytest.mark.parametrize("n", [31, 32, 33, 63, 64, 65])
def test_lines_that_end_at_the_lanes_of_a_warp(ts, d, last, n):
    """A warp looks 32 streams ahead: batches that end in front of its last lane, with
    it and behind it, with a stream that has nodes and with one that has none."""
    q, k = _streams(n, n, 64, 700)
    q[-1], k[-1] = last, 700
    b = pu.Batch(q, k, 4, 2, d, 32, BF, seed=n, extra=2)
    check(ts, b, parents_of(q, "mixed", seed=n, extra=2))


@pytest.mark.parametrize("kv", [64 + x for x in (0, 1, 31, 32, 33, 63, 64, 65, 96, 127, 128, 129)])
def test_every_place_in_a_tile(ts, kv):
    for dtype, Hq in ((BF, 4), (FP, 64)):
        b = pu.Batch([64] * 3, [kv] * 3, Hq, 1, 64, 16, dtype, seed=kv)
        check(ts, b, parents_of(b.q_lens, "any", seed=kv))


@pytest.mark.parametrize("Hq,kv", [(4, 300), (2, 40000), (8, 40000), (32, 40000)])
def test_other_branches_do_not_count(ts, Hq, kv):
    """Rows of other branches point along every query, far above the seen scores."""
    for dtype in (BF, FP):
        b = pu.Batch([64, 64], [kv, kv], Hq, 2, 128, 64, dtype, seed=5)
        par = parents_of([64, 64], "star")
        for s in range(2):
            for a in range(1, 64, 2):            # odd nodes: seen by themselves alone
                r = kv - 64 + a
                page = int(b.table_host[s, r // 64])
                b.k[page, :, r % 64] = 40.0
                b.v[page, :, r % 64] = 1000.0
        b.q.abs_()
        check(ts, b, par)


@pytest.mark.parametrize("Hq,kv", [(4, 500), (32, 30000)])
def test_chain_is_a_causal_chunk(ts, Hq, kv):
    b = pu.Batch([64, 20], [kv, kv], Hq, 2, 128, 32, BF, seed=6)
    o, lse = attend(ts, b, parents_of(b.q_lens, "chain"))
    o2, lse2 = ts.ts_paged_attention(b.q, b.k, b.v, b.cu_q, b.lens, b.table, 64)
    ref = oracle(b, parents_of(b.q_lens, "chain"))     # (the two may cut the keys elsewhere)
    pu.check_attention(o, lse, ref, BF, 128, p_round=P_ROUND[BF])
    pu.check_attention(o2, lse2, ref, BF, 128, p_round=P_ROUND[BF])


@pytest.mark.parametrize("Hq", [4, 8, 64])
def test_nodes_without_a_row(ts, Hq):
    """Lengths shorter than the trees: nodes whose rows and ancestors' are not there."""
    b = pu.Batch([40, 64, 5, 3], [40, 64, 5, 3], Hq, 2, 128, 16, BF, extra=1)
    par = parents_of(b.q_lens, "mixed", extra=1)
    b.kv_lens = [11, 1, 0, 3]
    b.lens = torch.tensor(b.kv_lens, dtype=torch.int32, device="cuda")
    o, lse = check(ts, b, par)
    assert (o[:29] == 0).all() and torch.isneginf(lse[:29]).all()
    assert (o[104:109] == 0).all()


@pytest.mark.parametrize("Hq,kv", [(4, 700), (2, 40000), (8, 20000), (64, 20000)])
@pytest.mark.parametrize("dtype", [BF, FP], ids=["bf16", "fp16"])
def test_large_scores(ts, Hq, kv, dtype):
    b = pu.Batch([64, 9], [kv, 90], Hq, 2, 128, 32, dtype, seed=9, scale=30.0)
    check(ts, b, parents_of(b.q_lens, "ternary"))


@pytest.mark.parametrize("Hq,kv", [(4, 300), (8, 20000), (64, 20000)])
@pytest.mark.parametrize("bad", [-1, -5, 30, 31, 10 ** 9])
def test_a_bad_parent_is_reported(ts, Hq, kv, bad):
    """Its node counts as a root; the other trees are as they should be."""
    b = pu.Batch([64, 64], [kv, kv], Hq, 2, 64, 32, BF, seed=10)
    par = parents_of(b.q_lens, "chain")
    ref = oracle(b, par)
    par[30] = bad
    o = torch.empty_like(b.q)
    lse = torch.empty(b.n, Hq, device="cuda")
    ts.ts_paged_tree_attention(b.q, b.k, b.v, b.cu_q, b.lens, b.table, par, 64, o=o, lse=lse,
                               status=b.status)
    assert status_of(b) == 1
    pu.check_attention(o[64:], lse[64:], tuple(x[64:] for x in ref), BF, 64, p_round=P_ROUND[BF])
    pu.check_attention(o[:30], lse[:30], tuple(x[:30] for x in ref), BF, 64, p_round=P_ROUND[BF])
    b.status.zero_()
    par[30], par[64] = 29, 0                      # a first node has no parent
    ts.ts_paged_tree_attention(b.q, b.k, b.v, b.cu_q, b.lens, b.table, par, 64, status=b.status)
    assert status_of(b) == 1


@pytest.mark.parametrize("Hq,kv", [(4, 300), (8, 20000), (64, 20000)])
def test_bad_pages_lengths_and_trees_are_reported(ts, Hq, kv):
    def call(b, max_q=64, **kw):
        b.status.zero_()
        ts.ts_paged_tree_attention(b.q, b.k, b.v, kw.get("cu", b.cu_q), kw.get("lens", b.lens),
                                   kw.get("table", b.table), par, max_q, o=o, lse=lse,
                                   status=b.status)
        return status_of(b)
    b = pu.Batch([64, 64], [kv, kv], Hq, 2, 64, 32, BF, seed=11)
    par = parents_of(b.q_lens, "any")
    o, lse = torch.empty_like(b.q), torch.empty(b.n, Hq, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    assert call(b) == 0
    assert call(b, max_q=63) == 1
    for page in (-3, 10 ** 9):
        table = b.table.clone()
        table[0, 2] = page
        assert call(b, table=table) == 1
        ref = tuple(x[64:] for x in oracle(b, par))
        pu.check_attention(o[64:], lse[64:], ref, BF, 64, p_round=P_ROUND[BF])
    for lens in ([10 ** 9, kv], [-4, kv]):
        assert call(b, lens=torch.tensor(lens, **i32)) == 1
    for cu in ([0, 64, 10 ** 6], [0, -5, 128], [0, 128, 128], [0, 90, 64]):
        assert call(b, cu=torch.tensor(cu, **i32)) == 1


@pytest.mark.parametrize("Hq,kv,q", [(4, 300, 64), (64, 20000, 64), (8, 20000, 64), (2, 90000, 64),
                                     (8, 60000, 5)])
def test_nan_in_a_query_row(ts, Hq, kv, q):
    b = pu.Batch([q, q], [kv, kv - 1], Hq, 2, 128, 32, FP, seed=19)
    par = parents_of(b.q_lens, "ternary")
    o, lse = attend(ts, b, par)
    t, h = q + q // 2, Hq - 2
    b.q[t, h, 3] = float("nan")
    o2, lse2 = attend(ts, b, par)
    assert torch.isnan(o2[t, h]).all() and torch.isnan(lse2[t, h])
    o2[t, h], lse2[t, h] = o[t, h], lse[t, h]
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("Hq,q", [(4, 5), (4, 64), (8, 64), (32, 64)])
def test_replay_sees_new_trees_and_lengths(ts, Hq, q):
    """Two graphs on one workspace, replayed on other lengths and parents."""
    b = pu.Batch([q, q], [15000, 7000], Hq, 2, 128, 16, BF, seed=15)
    par = parents_of(b.q_lens, "any")
    o, lse = torch.empty_like(b.q), torch.empty(b.n, Hq, device="cuda")
    need = ts.ts_paged_tree_attention_workspace_bytes(b.n, 2, Hq, 2, 128, b.table.shape[1], 16, q)
    ws = torch.empty(max(need, 256), dtype=torch.uint8, device="cuda")

    def call():
        ts.ts_paged_tree_attention(b.q, b.k, b.v, b.cu_q, b.lens, b.table, par, q, o=o, lse=lse,
                                   workspace=ws, status=b.status)
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        call()
    torch.cuda.synchronize()
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for g in graphs:
        with torch.cuda.graph(g):
            call()
    for i, lens in enumerate(([15000, 7000], [q, q + 1], [333, 164])):
        b.kv_lens = lens
        b.lens.copy_(torch.tensor(lens, dtype=torch.int32))
        par.copy_(parents_of(b.q_lens, "any", seed=i))
        ref = oracle(b, par)
        for g in graphs:
            o.zero_()
            g.replay()
            assert status_of(b) == 0
            pu.check_attention(o, lse, ref, BF, 128, p_round=P_ROUND[BF])


@pytest.mark.parametrize("Hq,q,kv", [(8, 3, 500), (8, 64, 2100), (40, 64, 30000)])
def test_another_stream_no_lse_and_repeatability(ts, Hq, q, kv):
    b = pu.Batch([q, q, q], [kv, 64, 800], Hq, 2, 128, 32, BF, seed=16)
    par = parents_of(b.q_lens, "ternary")
    o, lse = attend(ts, b, par)
    for _ in range(5):
        o2, lse2 = attend(ts, b, par)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    o2, lse2 = ts.ts_paged_tree_attention(b.q, b.k, b.v, b.cu_q, b.lens, b.table, par, q, stream=st)
    st.synchronize()
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    o2, none = ts.ts_paged_tree_attention(b.q, b.k, b.v, b.cu_q, b.lens, b.table, par, q,
                                          want_lse=False, max_kv=64)
    assert none is None
    pu.check_attention(o2, lse, oracle(b, par), BF, 128, p_round=P_ROUND[BF])


@pytest.mark.parametrize("q,Hq", [(5, 8), (64, 64)])
def test_pool_beyond_32_bit_offsets(ts, q, Hq):
    b = pu.Batch([q], [500], Hq, 8, 128, 128, BF, seed=18)
    n_pages = (1 << 32) // (8 * 128 * 128 * 2) + 40
    k = torch.zeros(n_pages, 8, 128, 128, dtype=BF, device="cuda")
    v = torch.zeros_like(k)
    far = torch.arange(n_pages - 4, n_pages, device="cuda")
    near = b.table[0, :4].long()
    k[far], v[far] = b.k[near], b.v[near]
    table = b.table.clone()
    table[0, :4] = far.int()
    par = parents_of([q], "any")
    o, lse = ts.ts_paged_tree_attention(b.q, k, v, b.cu_q, b.lens, table, par, q, status=b.status)
    assert status_of(b) == 0
    pu.check_attention(o, lse, oracle(b, par), BF, 128, p_round=P_ROUND[BF])
    # the accepted rows move there too
    path = torch.full((1, q), -2, dtype=torch.int32, device="cuda")
    path[0, :2] = torch.tensor([0, q - 1])
    n_path = torch.tensor([2], dtype=torch.int32, device="cuda")
    L = 500 - q
    want = k[far[(499) // 128], :, 499 % 128].clone()
    ts.ts_paged_kv_commit([k], [v], b.cu_q, b.lens, table, path, n_path, status=b.status)
    assert status_of(b) == 0
    assert torch.equal(k[far[(L + 1) // 128], :, (L + 1) % 128], want)


@pytest.mark.parametrize("Hq,kv", [(8, 30000), (2, 30000), (16, 30000)])
def test_an_expired_wait_is_reported(ts, Hq, kv):
    """A limit of a few clocks: a status, and the next call is as it should be."""
    b = pu.Batch([64, 64], [kv, kv - 77], Hq, 2, 128, 32, BF, seed=21)
    par = parents_of(b.q_lens, "any")
    o, lse = attend(ts, b, par)
    try:
        ts.ts_set_wait_limit(1)
        ts.ts_paged_tree_attention(b.q, b.k, b.v, b.cu_q, b.lens, b.table, par, 64, status=b.status)
        assert status_of(b) == 4
    finally:
        ts.ts_set_wait_limit(0)
    b.status.zero_()
    o2, lse2 = attend(ts, b, par)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_trees_on_two_streams_at_once(ts):
    batches = [pu.Batch([64] * 6, [9000 + 50 * i + k for i in range(6)], 8, 2, 128, 32, dt, seed=22 + k)
               for k, dt in enumerate((BF, FP))]
    pars = [parents_of(b.q_lens, "any", seed=k) for k, b in enumerate(batches)]
    refs = [attend(ts, b, p) for b, p in zip(batches, pars)]
    streams = [torch.cuda.Stream() for _ in batches]
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(8):
        for k, st in enumerate(streams):
            b = batches[k]
            outs[k].append(ts.ts_paged_tree_attention(b.q, b.k, b.v, b.cu_q, b.lens, b.table, pars[k],
                                                      64, status=b.status, stream=st))
    torch.cuda.synchronize()
    for k, (o, lse) in enumerate(refs):
        assert status_of(batches[k]) == 0
        for x, y in outs[k]:
            assert torch.equal(o, x) and torch.equal(lse, y)


def test_an_empty_batch(ts):
    b = pu.Batch([3], [3], 4, 2, 64, 16, BF)
    none = torch.empty(0, 4, 64, dtype=BF, device="cuda")
    cu = torch.zeros(2, dtype=torch.int32, device="cuda")
    par = torch.empty(0, dtype=torch.int32, device="cuda")
    o, lse = ts.ts_paged_tree_attention(none, b.k, b.v, cu, b.lens, b.table, par, 1)
    assert o.shape == (0, 4, 64) and lse.shape == (0, 4)


# ------------------------------------------------------------------ commit
def accepted(q_lens, seed=0, kind="any"):
    """Parents and, of every tree, a root path; [n_seq, T] and lengths."""
    rng = np.random.default_rng(seed)
    par, paths = [], []
    for n in q_lens:
        p = tree(kind, n, rng)
        par += p
        paths.append(po.root_paths(p)[int(rng.integers(0, n))] if n else [0])
    T = max(max(len(p) for p in paths), 1)
    path = torch.full((len(q_lens), T), -2, dtype=torch.int32)
    for s, p in enumerate(paths):
        path[s, :len(p)] = torch.tensor(p)
    return path.cuda(), torch.tensor([len(p) for p in paths], dtype=torch.int32, device="cuda")


def layers_of(b, n, seed=0):
    """n layers' pools over one table: finite rows everywhere."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    shape = (n, b.n_pages, b.Hkv, b.ps, b.d)
    return [torch.randn(shape, generator=g, device="cuda").to(b.dtype) for _ in range(2)]


def check_commit(ts, b, path, n_path, k, v, bounds, **kw):
    mn = mx = None
    if bounds:
        mn = (k.amin(3).float() - 1).to(b.dtype)
        mx = (k.amax(3).float() + 1).to(b.dtype)
        kw.update(key_min=mn, key_max=mx)
    refs = [po.kv_commit(pu.f64(k[i]), pu.f64(v[i]), pu.f64(mn[i]) if bounds else None,
                         pu.f64(mx[i]) if bounds else None, b.cu, b.kv_lens, b.table_host.numpy(),
                         path.cpu().numpy(), n_path.cpu().numpy()) for i in range(len(k))]
    new = ts.ts_paged_kv_commit(k, v, b.cu_q, b.lens, b.table, path, n_path, status=b.status, **kw)
    assert status_of(b) == 0
    assert new.tolist() == refs[0][4]
    for i, ref in enumerate(refs):
        np.testing.assert_array_equal(pu.f64(k[i]), ref[0])
        np.testing.assert_array_equal(pu.f64(v[i]), ref[1])
        if bounds:
            np.testing.assert_array_equal(pu.f64(mn[i]), ref[2])
            np.testing.assert_array_equal(pu.f64(mx[i]), ref[3])


@pytest.mark.parametrize("dtype", [BF, FP], ids=["bf16", "fp16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("ps", [16, 32, 64, 128])
def test_commit(ts, dtype, d, ps):
    for kind, bounds in (("any", True), ("ternary", False), ("chain", True)):
        b = pu.Batch([40, 0, 1, 64, 7, 33, 64], [100, 40, 300, 64, 7, 129, 1030], 4, 2, d, ps, dtype,
                     seed=ps)
        k, v = layers_of(b, 3, seed=ps)
        check_commit(ts, b, *accepted(b.q_lens, seed=ps, kind=kind), k, v, bounds)


@pytest.mark.parametrize("ps", [16, 128])
@pytest.mark.parametrize("L", [0, 1, 15, 16, 17, 127, 128])
def test_commit_across_pages(ts, ps, L):
    """Trees that start at every place of a page; the longest path, and a root alone."""
    b = pu.Batch([64, 64], [L + 64, L + 64], 2, 1, 64, ps, BF, seed=L)
    k, v = layers_of(b, 2, seed=L)
    path = torch.arange(64, dtype=torch.int32, device="cuda").repeat(2, 1)
    check_commit(ts, b, path, torch.tensor([64, 1], dtype=torch.int32, device="cuda"), k, v, True)
    jump = torch.tensor([[0, 9, 10, 40, 63]] * 2, dtype=torch.int32, device="cuda")
    check_commit(ts, b, jump, torch.tensor([5, 3], dtype=torch.int32, device="cuda"), k, v, True)


@pytest.mark.parametrize("Hkv,n", [(1, 1), (8, 32), (3, 7)])
def test_commit_lists_tables_and_streams(ts, Hkv, n):
    b = pu.Batch([5, 9], [50, 1000], Hkv, Hkv, 128, 32, BF, seed=3)
    path, n_path = accepted(b.q_lens, seed=1)
    k, v = layers_of(b, n)
    k2, v2 = [x.clone() for x in k], [x.clone() for x in v]
    check_commit(ts, b, path, n_path, k, v, False)
    table = ts.commit_pointer_table(k2, v2)
    new = torch.empty(2, dtype=torch.int32, device="cuda")
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    r = ts.ts_paged_kv_commit(k2, v2, b.cu_q, b.lens, b.table, path, n_path, table=table,
                              new_lens=new, stream=st)
    st.synchronize()
    assert r is new
    for i in range(n):
        assert torch.equal(k2[i], k[i]) and torch.equal(v2[i], v[i])


def test_commit_keeps_nan_and_other_bits(ts):
    """Rows are moved bit for bit; a NaN in a committed key shows in the bounds."""
    b = pu.Batch([4], [20], 1, 1, 64, 16, FP, seed=4)
    k, v = layers_of(b, 1)
    page = int(b.table_host[0, 1])
    k[0, page, 0, 3, 5] = float("nan")            # row 19, node 3
    v[0, page, 0, 3, 7] = float("inf")
    mn, mx = k.amin(3), k.amax(3)
    ts.ts_paged_kv_commit(k, v, b.cu_q, b.lens, b.table,
                          torch.tensor([[0, 3]], dtype=torch.int32, device="cuda"),
                          torch.tensor([2], dtype=torch.int32, device="cuda"), key_min=mn, key_max=mx,
                          status=b.status)
    assert status_of(b) == 0
    assert torch.equal(k[0, page, 0, 1].view(torch.int16), k[0, page, 0, 3].view(torch.int16))
    assert torch.isinf(v[0, page, 0, 1, 7]) and torch.isnan(mn[0, page, 0, 5])
    assert torch.isnan(mx[0, page, 0, 5]) and torch.isnan(mn[0, page]).sum() == 1


@pytest.mark.parametrize("path,m", [([0, 2, 1, 3], 4), ([0, 5, -1, 7], 4), ([0, 9, 3, 4], 3),
                                    ([0, 1, 2, 3], 0), ([0, 1, 2, 3], 5), ([0, 1, 2, 3], -2)])
def test_commit_reports_a_bad_path_and_moves_nothing(ts, path, m):
    b = pu.Batch([8, 8], [40, 50], 2, 1, 64, 16, BF, seed=5)
    k, v = layers_of(b, 2)
    k0, v0, mn = k.clone(), v.clone(), k.amin(3)
    mx, mn0 = k.amax(3), mn.clone()
    both = torch.tensor([[0, 3, 5, 6], path], dtype=torch.int32, device="cuda")
    n_path = torch.tensor([4, m], dtype=torch.int32, device="cuda")
    new = ts.ts_paged_kv_commit(k, v, b.cu_q, b.lens, b.table, both, n_path, key_min=mn, key_max=mx,
                                status=b.status)
    assert status_of(b) == 1 and new.tolist() == [36, 50]
    own = [int(p) for p in b.table_host[0, :3]]
    rest = [p for p in range(b.n_pages) if p not in own]
    assert torch.equal(k[:, rest], k0[:, rest]) and torch.equal(v[:, rest], v0[:, rest])
    assert torch.equal(mn[:, rest], mn0[:, rest])
    assert torch.equal(k[:, own[2], :, 33 - 32], k0[:, own[2], :, 35 - 32])


def test_commit_reports_bad_tables(ts):
    b = pu.Batch([8, 8], [40, 50], 2, 1, 64, 16, BF, seed=6)
    k, v = layers_of(b, 1)
    path = torch.tensor([[0, 3, 5, 6]] * 2, dtype=torch.int32, device="cuda")
    n_path = torch.tensor([4, 4], dtype=torch.int32, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    k0 = k.clone()
    for cu, lens, table in (([0, 8, 4], None, None), (None, [40, 10 ** 9], None), (None, [-1, 50], None),
                            (None, [5, 50], None), (None, None, -1), (None, None, 10 ** 9)):
        b.status.zero_()
        t = b.table.clone()
        if table is not None:
            t[0, 2] = table
        k.copy_(k0)
        ts.ts_paged_kv_commit(k, v, torch.tensor(cu, **i32) if cu else b.cu_q,
                              torch.tensor(lens, **i32) if lens else b.lens, t, path, n_path,
                              status=b.status)
        assert status_of(b) == 1


@pytest.mark.parametrize("what,cu,lens,page,at", [
    ("offset", [0, 8, 4], None, None, 1), ("offset", [0, 8, 2 ** 31 - 1], None, None, 1),
    ("offset", [-1, 8, 16], None, None, 0), ("length", None, [40, 10 ** 9], None, 1),
    ("length", None, [-1, 50], None, 0), ("short", None, [5, 50], None, 0),
    ("page", None, None, -1, 0), ("page", None, None, 10 ** 9, 0), ("page", None, None, 2 ** 31 - 1, 0)])
def test_commit_beside_bad_tables(ts, what, cu, lens, page, at):
    """The faulty stream's rows, bounds and length stay, the other's are committed."""
    b = pu.Batch([8, 8], [40, 50], 2, 2, 64, 16, BF, seed=6)
    k, v = layers_of(b, 3)
    mn, mx = (k.amin(3).float() - 1).to(BF), (k.amax(3).float() + 1).to(BF)
    path = torch.tensor([[0, 3, 5, 6]] * 2, dtype=torch.int32, device="cuda")
    n_path = torch.tensor([4, 4], dtype=torch.int32, device="cuda")
    table, cu, lens = b.table.clone(), cu or b.cu, lens or b.kv_lens
    if page is not None:
        table[0, 2] = page
    # the faulty stream as one without nodes
    good_cu = [0, 0, 8] if at == 0 else [0, 8, 8]
    refs = [po.kv_commit(*(pu.f64(x[i]) for x in (k, v, mn, mx)), good_cu, b.kv_lens,
                         b.table_host.numpy(), path.cpu().numpy(), [4, 4])
            for i in range(3)]
    i32 = dict(dtype=torch.int32, device="cuda")
    new = ts.ts_paged_kv_commit(k, v, torch.tensor(cu, **i32), torch.tensor(lens, **i32), table,
                                path, n_path, key_min=mn, key_max=mx, status=b.status)
    assert status_of(b) == 1
    want = list(lens)
    want[1 - at] = refs[0][4][1 - at]
    assert new.tolist() == want
    for i, ref in enumerate(refs):
        for x, r in zip((k, v, mn, mx), ref):
            np.testing.assert_array_equal(pu.f64(x[i]), r)


def test_commit_refuses_layers_that_start_off_a_boundary(ts):
    """The kernel takes the addresses from a table, where the library cannot see them."""
    b = pu.Batch([5], [20], 4, 2, 64, 16, BF)
    k, v = layers_of(b, 1)
    path, n_path = accepted(b.q_lens)
    off = torch.zeros(k.numel() + 8, dtype=BF, device="cuda")[4:4 + k.numel()].view(k.shape)
    mn, mx = k.amin(3), k.amax(3)
    off_bounds = torch.zeros(mn.numel() + 8, dtype=BF, device="cuda")[1:1 + mn.numel()].view(mn.shape)
    args = (b.cu_q, b.lens, b.table, path, n_path)
    for kp, vp, lo, hi in ((off, v, mn, mx), (k, off, mn, mx), ([k[0]], [off[0]], None, None),
                           (k, v, off_bounds, mx), (k, v, [mn[0]], [off_bounds[0]])):
        with pytest.raises(ValueError, match="aligned"):
            ts.ts_paged_kv_commit(kp, vp, *args, key_min=lo, key_max=hi)


@pytest.mark.parametrize("Hq,top,kv", [(8, 3, 300), (8, 64, 900), (32, 40, 5000), (64, 64, 5000)])
def test_sequences_of_a_larger_batch(ts, Hq, top, kv):
    """The last of a batch's sequences alone: the first offset is not 0."""
    b = pu.Batch([2, top, 1, top], [kv, kv, kv // 2, kv], Hq, 2, 128, 16, BF, seed=top, extra=3)
    par = parents_of(b.q_lens, "mixed", extra=3)
    want = oracle(b, par)
    for lead in (1, 2):
        o = torch.full((b.n, b.Hq, b.d), 55.0, dtype=b.dtype, device="cuda")
        lse = torch.full((b.n, b.Hq), 55.0, dtype=torch.float32, device="cuda")
        ts.ts_paged_tree_attention(b.q, b.k, b.v, b.cu_q[lead:].contiguous(),
                                   b.lens[lead:].contiguous(), b.table[lead:].contiguous(), par,
                                   top, o=o, lse=lse, status=b.status)
        assert status_of(b) == 0
        a, e = b.cu[lead], b.cu[-1]
        for x in (o, lse):
            assert (x[:a] == 55.0).all() and (x[e:] == 55.0).all()
        pu.check_attention(o[a:e], lse[a:e], tuple(x[a:e] for x in want), b.dtype, b.d,
                           p_round=P_ROUND[b.dtype])


def test_a_table_made_by_the_call_outlives_it_on_another_stream(ts, monkeypatch):
    b = pu.Batch([5], [20], 4, 2, 64, 16, BF)
    k, v = layers_of(b, 3)
    path, n_path = accepted(b.q_lens)
    new = torch.zeros(1, dtype=torch.int32, device="cuda")
    made, make = [], ts.commit_pointer_table

    def note(*a):
        t = make(*a)
        made.append(t.data_ptr())
        return t
    monkeypatch.setattr(ts, "commit_pointer_table", note)
    mn, mx = k.amin(3), k.amax(3)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(600_000_000)
    ts.ts_paged_kv_commit(k, v, b.cu_q, b.lens, b.table, path, n_path, key_min=mn, key_max=mx,
                          new_lens=new, status=b.status, stream=side)
    held = [torch.empty(2, 3, dtype=torch.int64, device="cuda") for _ in range(64)]
    waiting = not side.query()
    torch.cuda.synchronize()
    assert waiting and len(made) == 2
    assert not set(made) & {t.data_ptr() for t in held}
    assert status_of(b) == 0 and new.tolist() == [15 + int(n_path[0])]


def test_commit_replays_with_new_paths(ts):
    b = pu.Batch([16, 16], [200, 100], 2, 2, 128, 32, BF, seed=7)
    k, v = layers_of(b, 4)
    path, n_path = accepted(b.q_lens, seed=2, kind="chain")
    path = torch.cat([path, path.new_full((2, 16 - path.shape[1]), -2)], 1)
    table, new = ts.commit_pointer_table(k, v), torch.zeros(2, dtype=torch.int32, device="cuda")

    def call():
        ts.ts_paged_kv_commit(k, v, b.cu_q, b.lens, b.table, path, n_path, table=table,
                              new_lens=new, status=b.status)
    st = torch.cuda.Stream()
    n_path.fill_(1)
    with torch.cuda.stream(st):
        call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for i in range(3):
        p, m = accepted(b.q_lens, seed=10 + i)
        path.fill_(-2)
        path[:, :p.shape[1]] = p
        n_path.copy_(m)
        refs = [po.kv_commit(pu.f64(k[j]), pu.f64(v[j]), None, None, b.cu, b.kv_lens,
                             b.table_host.numpy(), path.cpu().numpy(), m.cpu().numpy())
                for j in range(4)]
        g.replay()
        assert status_of(b) == 0 and new.tolist() == refs[0][4]
        for j in range(4):
            np.testing.assert_array_equal(pu.f64(k[j]), refs[j][0])
            np.testing.assert_array_equal(pu.f64(v[j]), refs[j][1])
