"""GPU parity of the paged-cache operators against the 64-bit oracle: the
rotary append, attention over pages, the choice of pages, attention over
chosen pages, and a run of them together."""
import numpy as np
import pytest
import torch

from oracle import paged_oracle as po
import paged_util as pu

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16
# weights P enter P.V as a 16-bit value and its 16-bit remainder where the
# rows are few, as one 16-bit value where tiles of rows are (half a step)
P_ROUND = {BF: 2.0 ** -8, FP: 2.0 ** -11}


@pytest.fixture(scope="module")
def ts():
    import self_speculative_ultra_gb300 as ts
    ts.build()
    return ts


def status_of(b):
    torch.cuda.synchronize()
    return int(b.status.item())


# ------------------------------------------------------------------ append
def _append_case(ts, q_lens, kv_lens, Hq, Hkv, d, ps, dtype, rot, inter, factor=1.0, tree=False,
                 bounds=True, seed=0, extra=0, far=0):
    b = pu.Batch(q_lens, kv_lens, Hq, Hkv, d, ps, dtype, seed=seed, extra=extra)
    g = torch.Generator().manual_seed(seed + 1)
    # rows of a fused projection: q, k and v of a token side by side
    x = torch.randn(max(b.n, 1), (Hq + 2 * Hkv) * d, generator=g).to(dtype).cuda()[:b.n]
    q = x[:, :Hq * d].view(b.n, Hq, d)
    k = x[:, Hq * d:(Hq + Hkv) * d].view(b.n, Hkv, d)
    v = x[:, (Hq + Hkv) * d:].view(b.n, Hkv, d)
    freqs, scale = ts.ts_rope_frequencies(rot, scaling="ramp" if factor > 1 else "plain",
                                          factor=factor, original_len=4096.0) if rot else \
        (torch.zeros(0, dtype=torch.float64, device="cuda"), 1.0)
    places = po.token_rows(b.cu, b.kv_lens)
    rng = np.random.default_rng(seed)
    pos = np.zeros(b.n, dtype=np.int32)
    for t, s, p in places:
        pos[t] = p + far - (int(rng.integers(0, 3)) if tree else 0)
    positions = torch.from_numpy(pos).cuda() if (tree or far) else None
    k0, v0 = b.k.clone(), b.v.clone()
    kmin = torch.randn(b.n_pages, Hkv, d, generator=g).to(dtype).cuda() if bounds else None
    kmax = (kmin + 1.0).to(dtype) if bounds else None
    mn0, mx0 = (kmin.clone(), kmax.clone()) if bounds else (None, None)
    q_out = torch.full((b.n, Hq, d), 77.0, dtype=dtype, device="cuda")
    r = ts.ts_paged_rope_append(q, k, v, b.cu_q, b.lens, b.table, b.k, b.v, freqs,
                                positions=positions, rope_scale=scale, interleaved=inter,
                                key_min=kmin, key_max=kmax, q_out=q_out, status=b.status)
    assert r is q_out and status_of(b) == 0
    fr = freqs.cpu().numpy()
    written = {}
    Q, K, got_q = pu.f64(q), pu.f64(k), pu.f64(q_out)
    u, tiny = pu.U[dtype], pu.TINY[dtype]

    def near(got, src, t):
        ref = po.rotate_row(src, float(pos[t]), fr, scale, inter)
        # the angle's fraction of a turn is off by a few 2^-24, times 2 pi;
        # cos, sin, two products and a sum add a few 2^-24 more: 2^-19 of the pair
        mag = np.abs(src) + np.abs(src).max()
        delta = 2.0 ** -19 * mag * scale
        assert (np.abs(got - ref) <= u * (np.abs(ref) + delta) + delta + tiny).all()
        r2 = 2 * len(fr)
        np.testing.assert_array_equal(got[..., r2:], src[..., r2:])

    for t, s, p in places:
        near(got_q[t], Q[t], t)
        written[(int(b.table_host[s, p // ps]), p % ps)] = t
    assert (got_q[b.cu[-1]:] == 77.0).all()          # rows behind the last sequence
    gk = pu.f64(b.k)
    for (page, row), t in written.items():
        near(gk[page, :, row], K[t], t)
        assert torch.equal(b.v[page, :, row], v[t])
    # nothing else moved (bit patterns: unowned rows are NaN)
    keep = torch.ones(b.n_pages, ps, dtype=torch.bool)
    for page, row in written:
        keep[page, row] = False
    keep = keep.cuda()
    for new, old in ((b.k, k0), (b.v, v0)):
        a, c = (y.view(torch.int16).permute(0, 2, 1, 3)[keep] for y in (new, old))
        assert torch.equal(a, c)
    if bounds:
        pages = {}
        for page, row in written:
            pages.setdefault(page, []).append(row)
        for page, rows in pages.items():
            x = b.k[page][:, sorted(rows)]
            mn, mx = x.amin(1), x.amax(1)
            if min(rows) > 0:
                mn, mx = torch.minimum(mn, mn0[page]), torch.maximum(mx, mx0[page])
                mn, mx = torch.minimum(mn, mx0[page]), torch.maximum(mx, mn0[page])
            assert torch.equal(kmin[page], mn) and torch.equal(kmax[page], mx)
        rest = [p for p in range(b.n_pages) if p not in pages]
        assert torch.equal(kmin[rest], mn0[rest]) and torch.equal(kmax[rest], mx0[rest])


@pytest.mark.parametrize("dtype", [BF, FP], ids=["bf16", "fp16"])
@pytest.mark.parametrize("d,rot,inter", [(128, 128, False), (128, 64, True), (128, 48, False),
                                         (64, 64, False), (64, 16, True), (64, 0, False)])
@pytest.mark.parametrize("ps", [16, 64])
def test_append_layouts(ts, dtype, d, rot, inter, ps):
    _append_case(ts, [5, 0, 70, 1, 33], [5, 9, 133, 64, 40], 4, 2, d, ps, dtype, rot, inter,
                 extra=3)


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (12, 2), (40, 8), (7, 7), (36, 12)])
@pytest.mark.parametrize("ps", [32, 128])
def test_append_head_counts(ts, Hq, Hkv, ps):
    _append_case(ts, [1, 17, 200], [33, 17, 1000], Hq, Hkv, 128, ps, BF, 128, False, seed=3)


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (8, 8), (32, 4)])
def test_append_small_heads_in_long_pages(ts, Hq, Hkv):
    """Few units a head row: a thread's token lanes outnumber a trip's tokens."""
    _append_case(ts, [130, 128, 1], [130, 300, 128], Hq, Hkv, 64, 128, BF, 64, False, seed=4)


@pytest.mark.parametrize("n_seq", [1, 255, 256, 700])
def test_append_many_single_tokens(ts, n_seq):
    kv = [(37 * s) % 50 + 1 for s in range(n_seq)]
    _append_case(ts, [1] * n_seq, kv, 4, 2, 64, 16, BF, 64, False, seed=n_seq)


def test_append_long_prompt_fills_many_blocks(ts):
    _append_case(ts, [3000, 1], [3000, 2], 8, 4, 128, 64, FP, 128, False, bounds=True, seed=5)


@pytest.mark.parametrize("far", [100000, (1 << 24) + 12345, (1 << 29) + 7, -5000])
def test_append_far_positions(ts, far):
    _append_case(ts, [9, 4], [9, 30], 4, 1, 128, 16, FP, 128, False, far=far, seed=6)


def test_append_tree_positions_and_scaled_frequencies(ts):
    _append_case(ts, [64], [300], 16, 4, 128, 64, BF, 128, False, factor=8.0, tree=True, seed=7)
    _append_case(ts, [64], [300], 16, 4, 128, 64, BF, 128, True, bounds=False, seed=8)


def test_append_in_place_queries_and_dense_inputs(ts):
    b = pu.Batch([40, 3], [40, 9], 4, 2, 128, 32, BF)
    k, v = (torch.randn(b.n, 2, 128, device="cuda").to(BF) for _ in range(2))
    freqs, _ = ts.ts_rope_frequencies(128)
    kp, vp = b.k.clone(), b.v.clone()
    out = ts.ts_paged_rope_append(b.q, k, v, b.cu_q, b.lens, b.table, kp, vp, freqs)
    q = b.q.clone()
    r = ts.ts_paged_rope_append(q, k, v, b.cu_q, b.lens, b.table, b.k, b.v, freqs, q_out=q)
    assert r is q and torch.equal(q, out)
    assert torch.equal(kp.view(torch.int16), b.k.view(torch.int16))


@pytest.mark.parametrize("bad", [-1, 10 ** 9])
def test_append_reports_a_bad_page_and_leaves_it_alone(ts, bad):
    b = pu.Batch([3, 20], [3, 20], 4, 2, 64, 16, BF)
    b.table[0, 0] = bad
    k, v = (torch.randn(b.n, 2, 64, device="cuda").to(BF) for _ in range(2))
    freqs, _ = ts.ts_rope_frequencies(64)
    k0 = b.k.clone()
    ts.ts_paged_rope_append(b.q, k, v, b.cu_q, b.lens, b.table, b.k, b.v, freqs, status=b.status)
    assert status_of(b) == 1
    good = [int(p) for p in b.table_host[1, :2]]
    rest = [p for p in range(b.n_pages) if p not in good]
    assert torch.equal(b.k[rest].view(torch.int16), k0[rest].view(torch.int16))
    assert torch.equal(b.v[good[0], :, 5], v[3 + 5])


@pytest.mark.parametrize("lens,cu", [([3, 10 ** 9], None), ([-4, 20], None), ([2, 20], None),
                                     (None, [0, 3, 10 ** 6]), (None, [0, -5, 23]),
                                     (None, [0, 9, 3])])
def test_tables_out_of_range_are_reported(ts, lens, cu):
    """Lengths and token offsets outside their range: a status, and no access
    outside the buffers (the same clamps serve every call)."""
    b = pu.Batch([3, 20], [3, 20], 4, 2, 64, 16, BF)
    if lens:
        b.lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
    if cu:
        b.cu_q = torch.tensor(cu, dtype=torch.int32, device="cuda")
    k, v = (torch.randn(b.n, 2, 64, device="cuda").to(BF) for _ in range(2))
    freqs, _ = ts.ts_rope_frequencies(64)
    ts.ts_paged_rope_append(b.q, k, v, b.cu_q, b.lens, b.table, b.k, b.v, freqs, status=b.status)
    assert status_of(b) == 1
    if lens == [2, 20]:
        return              # fewer rows than new tokens: attention has rows without keys
    b.status.zero_()
    ts.ts_paged_attention(b.q, b.k, b.v, b.cu_q, b.lens, b.table, max_q=20, status=b.status)
    assert status_of(b) == 1


# ------------------------------------------------------------------ attention
def _attend(ts, b, **kw):
    o = torch.full((b.n, b.Hq, b.d), 55.0, dtype=b.dtype, device="cuda")
    lse = torch.full((b.n, b.Hq), 55.0, dtype=torch.float32, device="cuda")
    kw.setdefault("max_q", b.max_q)
    ts.ts_paged_attention(b.q, b.k, b.v, b.cu_q, b.lens, b.table, o=o, lse=lse, status=b.status,
                          **kw)
    assert status_of(b) == 0
    end = b.cu[-1]
    assert (o[end:] == 55.0).all() and (lse[end:] == 55.0).all()
    return o, lse


def _check_attend(ts, b, **kw):
    o, lse = _attend(ts, b, **kw)
    pu.check_attention(o, lse, b.oracle(), b.dtype, b.d, p_round=P_ROUND[b.dtype])
    return o, lse


@pytest.mark.parametrize("dtype", [BF, FP], ids=["bf16", "fp16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("ps", [16, 32, 64, 128])
def test_decode(ts, dtype, d, ps):
    b = pu.Batch([1] * 7, [1, 15, 16, 17, 129, 1000, 2500], 8, 2, d, ps, dtype, seed=ps, extra=2)
    _check_attend(ts, b)


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (8, 8), (12, 2), (40, 8), (16, 1), (24, 1), (17, 1)])
def test_decode_head_groups(ts, Hq, Hkv):
    b = pu.Batch([1, 1, 1], [300, 1, 77], Hq, Hkv, 128, 16, BF, seed=Hq)
    _check_attend(ts, b)


@pytest.mark.parametrize("dtype", [BF, FP], ids=["bf16", "fp16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("ps", [16, 32, 64, 128])
def test_chunks(ts, dtype, d, ps):
    """Prompts, chunks behind a cache, single tokens, sequences without new
    tokens and an empty sequence in one call."""
    b = pu.Batch([130, 0, 1, 64, 257, 0, 3], [130, 40, 300, 500, 258, 0, 3], 4, 2, d, ps, dtype,
                 seed=10 + ps, extra=5)
    _check_attend(ts, b)


@pytest.mark.parametrize("Hq,Hkv", [(2, 2), (5, 1), (12, 2), (40, 8), (16, 1)])
@pytest.mark.parametrize("q,kv", [(2, 2), (37, 400), (129, 129), (300, 1111)])
def test_chunk_head_groups(ts, Hq, Hkv, q, kv):
    b = pu.Batch([q, q // 2], [kv, kv], Hq, Hkv, 128, 64, BF, seed=Hq + q)
    _check_attend(ts, b)


def test_tokens_without_a_key_get_zero(ts):
    """Lengths shorter than the new tokens leave rows with nothing to see."""
    b = pu.Batch([4, 40, 3, 1], [4, 40, 3, 1], 4, 2, 128, 16, BF, extra=1)
    b.kv_lens = [2, 11, 0, 0]
    b.lens = torch.tensor(b.kv_lens, dtype=torch.int32, device="cuda")
    o, lse = _check_attend(ts, b)
    assert (o[4:4 + 29] == 0).all() and torch.isneginf(lse[4:4 + 29]).all()
    b = pu.Batch([400, 90], [400, 90], 16, 2, 128, 16, BF, extra=1)      # tiles of rows
    b.kv_lens = [130, 0]
    b.lens = torch.tensor(b.kv_lens, dtype=torch.int32, device="cuda")
    o, lse = _check_attend(ts, b)
    assert (o[:270] == 0).all() and (o[400:490] == 0).all()
    b = pu.Batch([1, 1], [1, 30], 4, 2, 64, 16, FP)
    b.kv_lens = [0, 30]
    b.lens = torch.tensor(b.kv_lens, dtype=torch.int32, device="cuda")
    _check_attend(ts, b)


@pytest.mark.parametrize("q", [1, 50, 600])
def test_large_scores(ts, q):
    """Scores of hundreds: the running maximum moves, old sums rescale."""
    b = pu.Batch([q, q], [700, 90], 4, 2, 128, 32, BF, seed=9, scale=30.0)
    _check_attend(ts, b)
    b = pu.Batch([q, q], [700, 90], 4, 2, 128, 32, FP, seed=9, scale=30.0)
    _check_attend(ts, b)


@pytest.mark.parametrize("q", [1, 30, 200])
def test_host_bound_on_lengths_is_only_a_hint(ts, q):
    b = pu.Batch([q] * 2, [3000, 40], 4, 2, 128, 16, BF, seed=11)
    o, lse = _check_attend(ts, b, max_kv=64)
    o2, lse2 = _check_attend(ts, b, max_kv=2999)


def test_tiles_with_a_short_hint(ts):
    """Tiles of rows where the host's bound is far below the lengths."""
    b = pu.Batch([160] * 8, [300, 200, 160, 1000, 170, 290, 900, 161], 16, 1, 64, 16, FP, seed=45)
    _check_attend(ts, b, max_kv=64)


@pytest.mark.parametrize("q", [1, 33, 150])
def test_without_lse_and_with_a_workspace(ts, q):
    b = pu.Batch([q] * 3, [900, 33, 2000], 8, 2, 64, 64, FP, seed=12)
    o, lse = _attend(ts, b)
    need = ts.ts_paged_attention_workspace_bytes(b.n, 3, 8, 2, 64, b.table.shape[1], 64, q)
    ws = torch.full((max(need, 1) + 256,), 255, dtype=torch.uint8, device="cuda")
    ws = ws[(-ws.data_ptr()) % 256:][:max(need, 1)]
    o2, none = ts.ts_paged_attention(b.q, b.k, b.v, b.cu_q, b.lens, b.table, q, want_lse=False,
                                     workspace=ws)
    assert none is None and torch.equal(o, o2)


@pytest.mark.parametrize("q,Hq", [(1, 4), (40, 4), (150, 32)])
def test_attention_reports_a_bad_page(ts, q, Hq):
    b = pu.Batch([q, q], [300, 300], Hq, 2, 128, 16, BF, seed=13)
    ref = b.oracle()
    b.table[0, 3] = -7
    o = torch.empty_like(b.q)
    lse = torch.empty(b.n, Hq, device="cuda")
    ts.ts_paged_attention(b.q, b.k, b.v, b.cu_q, b.lens, b.table, q, o=o, lse=lse, status=b.status)
    assert status_of(b) == 1
    # the other sequence is as it should be
    pu.check_attention(o[q:], lse[q:], tuple(x[q:] for x in ref), BF, 128, p_round=P_ROUND[BF])


def test_more_new_tokens_than_announced_is_reported(ts):
    b = pu.Batch([5, 1], [50, 60], 4, 2, 64, 16, BF, seed=14)
    o, lse = torch.empty_like(b.q), torch.empty(b.n, 4, device="cuda")
    ts.ts_paged_attention(b.q, b.k, b.v, b.cu_q, b.lens, b.table, 1, o=o, lse=lse, status=b.status)
    assert status_of(b) == 1


@pytest.mark.parametrize("q", [1, 24, 300])
def test_replay_sees_new_lengths(ts, q):
    """A captured call reads lengths, offsets and tables when it is replayed,
    and two graphs may run after one another on one workspace."""
    b = pu.Batch([q, q], [1500, 700], 4, 2, 128, 16, BF, seed=15)
    o, lse = torch.empty_like(b.q), torch.empty(b.n, 4, device="cuda")
    need = ts.ts_paged_attention_workspace_bytes(b.n, 2, 4, 2, 128, b.table.shape[1], 16, q)
    ws = torch.empty(max(need, 256), dtype=torch.uint8, device="cuda")

    def call():
        ts.ts_paged_attention(b.q, b.k, b.v, b.cu_q, b.lens, b.table, q, o=o, lse=lse,
                              workspace=ws, status=b.status)
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        call()
    torch.cuda.synchronize()
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for g in graphs:
        with torch.cuda.graph(g):
            call()
    for lens in ([1500, 700], [q, 1], [333, 164]):
        b.kv_lens = lens
        b.lens.copy_(torch.tensor(lens, dtype=torch.int32))
        for g in graphs:
            o.zero_()
            g.replay()
            assert status_of(b) == 0
            pu.check_attention(o, lse, b.oracle(), BF, 128, p_round=P_ROUND[BF])


@pytest.mark.parametrize("q", [1, 40, 300])
def test_another_stream_and_repeatability(ts, q):
    b = pu.Batch([q, q, q], [2100, max(q, 64), 800], 8, 2, 128, 32, BF, seed=16)
    o, lse = _attend(ts, b)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    o2, lse2 = ts.ts_paged_attention(b.q, b.k, b.v, b.cu_q, b.lens, b.table, q, stream=st)
    st.synchronize()
    assert torch.equal(o, o2) and torch.equal(lse, lse2)      # same bits every time


@pytest.mark.parametrize("d", [64, 128])
def test_same_bits_where_tiles_are_cut(ts, d):
    """Many tiles of nearly one cost: which are cut, and where, is always the same."""
    lens = [9000 + 37 * i % 150 for i in range(24)]
    b = pu.Batch([320] * 24, lens, 8, 2, d, 64, BF, seed=18)
    o, lse = _attend(ts, b)
    for _ in range(12):
        o2, lse2 = _attend(ts, b)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("q,kv,Hq,Hkv,d", [(1, 300, 8, 2, 64),       # a cluster a unit
                                           (1, 60000, 8, 2, 128),    # units cut in stretches
                                           (200, 600, 12, 2, 64),    # short tiles
                                           (200, 600, 12, 2, 128),
                                           (300, 30000, 12, 2, 64),  # cut tiles
                                           (300, 30000, 12, 2, 128)])
def test_nan_in_a_query_row(ts, q, kv, Hq, Hkv, d):
    """It reaches that row's o and lse, however the keys are split, and no other."""
    b = pu.Batch([q, q], [kv, kv - 1], Hq, Hkv, d, 32, BF, seed=19)
    o, lse = _attend(ts, b)
    t, h = q + q // 2, Hq - 2
    b.q[t, h, 3] = float("nan")
    o2, lse2 = _attend(ts, b)
    assert torch.isnan(o2[t, h]).all() and torch.isnan(lse2[t, h])
    o2[t, h], lse2[t, h] = o[t, h], lse[t, h]
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_nan_in_a_query_row_over_chosen_pages(ts):
    b = pu.Batch([1, 1], [900, 5000], 8, 2, 128, 32, BF, seed=20)
    pages = torch.arange(20, dtype=torch.int32, device="cuda").expand(2, 2, 20).contiguous()
    counts = torch.full((2, 2), 20, dtype=torch.int32, device="cuda")
    call = lambda: ts.ts_paged_attention_selected(  # noqa: E731
        b.q, b.k, b.v, b.cu_q, b.lens, b.table, pages, counts, status=b.status)
    o, lse = call()
    b.q[1, 5, 9] = float("nan")
    o2, lse2 = call()
    assert status_of(b) == 0 and torch.isnan(o2[1, 5]).all() and torch.isnan(lse2[1, 5])
    o2[1, 5], lse2[1, 5] = o[1, 5], lse[1, 5]
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("q,Hq,Hkv,d", [(1, 2, 1, 64), (40, 2, 1, 64), (1, 5, 1, 128), (33, 4, 1, 128)])
def test_long_cache(ts, q, Hq, Hkv, d):
    """Hundreds of thousands of rows: many splits, pieces and partial sums."""
    b = pu.Batch([q], [260_003], Hq, Hkv, d, 64, BF, seed=17)
    _check_attend(ts, b)


@pytest.mark.parametrize("q,Hq", [(1, 8), (30, 8), (130, 32)])
def test_pool_beyond_32_bit_offsets(ts, q, Hq):
    """Pages whose bytes lie past 2^32: offsets are 64-bit in every kernel."""
    b = pu.Batch([q], [500], Hq, 8, 128, 128, BF, seed=18)
    n_pages = (1 << 32) // (8 * 128 * 128 * 2) + 40            # 4.3 GB a tensor
    k = torch.zeros(n_pages, 8, 128, 128, dtype=BF, device="cuda")
    v = torch.zeros_like(k)
    far = torch.arange(n_pages - 4, n_pages, device="cuda")
    near = b.table[0, :4].long()
    k[far], v[far] = b.k[near], b.v[near]
    table = b.table.clone()
    table[0, :4] = far.int()
    ref = b.oracle()
    o, lse = ts.ts_paged_attention(b.q, k, v, b.cu_q, b.lens, table, q, status=b.status)
    assert status_of(b) == 0
    pu.check_attention(o, lse, ref, BF, 128, p_round=P_ROUND[BF])
    pages = torch.arange(4, dtype=torch.int32, device="cuda").expand(q, 8, 4).contiguous()
    counts = torch.full((q, 8), 4, dtype=torch.int32, device="cuda")
    rows = torch.arange(500 - q, 500, device="cuda")
    counts = (rows // 128 + 1).int()[:, None].expand(q, 8).contiguous()
    o, lse = ts.ts_paged_attention_selected(b.q, k, v, b.cu_q, b.lens, table, pages, counts,
                                            status=b.status)
    assert status_of(b) == 0
    pu.check_attention(o, lse, ref, BF, 128)
    mn, mx = k[far].amin(2), k[far].amax(2)
    kmin, kmax = (torch.zeros(n_pages, 8, 128, dtype=BF, device="cuda") for _ in range(2))
    freqs, _ = ts.ts_rope_frequencies(128)
    x = torch.randn(q, 8, 128, device="cuda").to(BF)
    ts.ts_paged_rope_append(b.q, x, x, b.cu_q, b.lens, table, k, v, freqs, key_min=kmin,
                            key_max=kmax, status=b.status)
    assert status_of(b) == 0
    slot = torch.arange(500 - q, 500, device="cuda")
    assert torch.equal(v[far[slot // 128], :, slot % 128], x)
    assert (kmax[far[3]] >= k[far[3], :, :500 - 384].amax(1)).all() or q < 116


@pytest.mark.parametrize("q", [1, 300])
def test_sequences_that_share_pages(ts, q):
    """Two sequences with the same first pages (a common prefix) and their own
    last ones."""
    b = pu.Batch([q, q], [640, 700], 8, 2, 128, 64, BF, seed=19)
    b.table[1, :5] = b.table[0, :5]
    b.table_host = b.table.cpu()
    _check_attend(ts, b)


@pytest.mark.parametrize("q", [1, 20, 150])
def test_two_streams_at_once(ts, q):
    """Calls on two streams, each with its own memory, while both run."""
    bs = [pu.Batch([q] * 4, [3000, 900, 2500, 700], 8, 2, 128, 32, BF, seed=s) for s in (42, 43)]
    want = [_attend(ts, b) for b in bs]
    streams = [torch.cuda.Stream() for _ in bs]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(6):
        for i, b in enumerate(bs):
            got[i].append(ts.ts_paged_attention(b.q, b.k, b.v, b.cu_q, b.lens, b.table, q,
                                                stream=streams[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for o, lse in got[i]:
            assert torch.equal(o, want[i][0]) and torch.equal(lse, want[i][1])


@pytest.mark.parametrize("d", [64, 128])
def test_short_wait_limit_and_the_call_behind_it(ts, d):
    """With a limit of a few clocks the chunk kernel gives up a wait that
    outlasts one hardware attempt, reports it, ends its copies and products and
    returns; waits that end within an attempt leave a right result."""
    b = pu.Batch([200], [900], 32, 2, d, 32, BF, seed=44)
    ref = b.oracle()
    ts.ts_set_wait_limit(1)
    try:
        o, lse = ts.ts_paged_attention(b.q, b.k, b.v, b.cu_q, b.lens, b.table, 200,
                                       status=b.status)
        torch.cuda.synchronize()
    finally:
        ts.ts_set_wait_limit(0)
    assert status_of(b) in (0, 4)
    if status_of(b) == 0:
        pu.check_attention(o, lse, ref, BF, d, p_round=P_ROUND[BF])
    b.status.zero_()
    _check_attend(ts, b)


def test_batch_of_nothing(ts):
    """No new token anywhere, and no sequence at all."""
    b = pu.Batch([0, 0], [40, 0], 4, 2, 64, 16, BF, extra=3)
    o = torch.full_like(b.q, 5.0)
    ts.ts_paged_attention(b.q, b.k, b.v, b.cu_q, b.lens, b.table, 1, o=o, want_lse=False,
                          status=b.status)
    ts.ts_paged_attention(b.q, b.k, b.v, b.cu_q, b.lens, b.table, 3, o=o, want_lse=False,
                          status=b.status)
    x = torch.zeros(3, 2, 64, dtype=BF, device="cuda")
    k0 = b.k.clone()
    freqs, _ = ts.ts_rope_frequencies(64)
    ts.ts_paged_rope_append(b.q, x, x, b.cu_q, b.lens, b.table, b.k, b.v, freqs, q_out=o,
                            status=b.status)
    assert status_of(b) == 0
    assert (o == 5.0).all() and torch.equal(k0.view(torch.int16), b.k.view(torch.int16))
    none = b.q[:0]
    o, lse = ts.ts_paged_attention(none, b.k, b.v, torch.zeros(1, dtype=torch.int32, device="cuda"),
                                   b.lens[:0], b.table[:0], 1)
    assert o.shape == (0, 4, 64) and lse.shape == (0, 4)


# ------------------------------------------------------------------ choice of pages
def _bounds(b, seed=0, grid=None):
    g = torch.Generator().manual_seed(seed)
    mid = torch.randn(b.n_pages, b.Hkv, b.d, generator=g)
    half = torch.rand(b.n_pages, b.Hkv, b.d, generator=g)
    if grid:
        mid, half = (mid / grid).round() * grid, (half / grid).round() * grid
    return (mid - half).to(b.dtype).cuda(), (mid + half).to(b.dtype).cuda()


def _check_select(ts, b, n_top, n_sink, n_recent, mn, mx):
    N = n_top + n_sink + n_recent
    pages = torch.full((b.n, b.Hkv, N), -7, dtype=torch.int32, device="cuda")
    counts = torch.full((b.n, b.Hkv), -7, dtype=torch.int32, device="cuda")
    ts.ts_paged_select_pages(b.q, mn, mx, b.cu_q, b.lens, b.table, b.ps, n_top, n_sink, n_recent,
                             pages=pages, counts=counts, status=b.status)
    assert status_of(b) == 0
    P, C = po.select_pages(pu.f64(b.q), pu.f64(mn), pu.f64(mx), b.cu, b.kv_lens,
                           b.table_host.numpy(), b.ps, n_top, n_sink, n_recent)
    np.testing.assert_array_equal(counts.cpu().numpy(), C)
    np.testing.assert_array_equal(pages.cpu().numpy(), P)
    return pages, counts


@pytest.mark.parametrize("dtype", [BF, FP], ids=["bf16", "fp16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq,Hkv", [(4, 4), (12, 2), (16, 1)])
def test_select(ts, dtype, d, Hq, Hkv):
    b = pu.Batch([1, 1, 5, 0, 1], [1, 400, 2000, 70, 3300], Hq, Hkv, d, 16, dtype, seed=20, extra=2)
    mn, mx = _bounds(b, 21)
    for top, sink, recent in ((8, 1, 2), (1, 0, 1), (0, 2, 3), (100, 0, 1), (300, 4, 4)):
        _check_select(ts, b, top, sink, recent, mn, mx)


def test_select_ties_go_to_the_lowest_page(ts):
    b = pu.Batch([1, 3], [5000, 4000], 4, 2, 64, 16, BF, seed=22)
    b.q = (b.q / 2).round().to(BF) * 2         # coarse values: sums are exact, ties many
    mn, mx = _bounds(b, 23, grid=1.0)
    for top in (1, 7, 100):
        _check_select(ts, b, top, 1, 1, mn, mx)
    zero = torch.zeros_like(mn)
    _check_select(ts, b, 9, 1, 2, zero, zero)  # every score equal


@pytest.mark.parametrize("dtype", [BF, FP], ids=["bf16", "fp16"])
@pytest.mark.parametrize("d", [64, 128])
def test_select_scores_close_to_the_cut(ts, dtype, d):
    """Pages that differ from one another by a step of one bound: the sums lie
    within fp32's rounding of each other, and only well formed ones rank them."""
    b = pu.Batch([1, 2], [6000, 2500], 6, 2, d, 16, dtype, seed=34)
    mn, mx = _bounds(b, 35)
    g = torch.Generator().manual_seed(36)
    one = mx[:1].clone()
    mx[:] = one
    mn[:] = mn[:1].clone()
    # every page: one column of the maximum a step or two away
    col = torch.randint(0, d, (b.n_pages, 2), generator=g).cuda()
    step = (1 + torch.randint(0, 2, (b.n_pages, 2), generator=g).cuda()).to(torch.int16)
    bits = mx.view(torch.int16)
    pg = torch.arange(b.n_pages, device="cuda")[:, None].expand(-1, 2)
    hd = torch.arange(2, device="cuda")[None, :].expand(b.n_pages, -1)
    bits[pg, hd, col] = bits[pg, hd, col] + step
    small = (b.q.float() * 0.003).to(dtype)
    b.q = torch.where(torch.rand(b.q.shape, generator=g).cuda() < 0.7, small, b.q)
    for top in (1, 30, 100):
        _check_select(ts, b, top, 1, 1, mn, mx)


def test_select_scores_that_cancel(ts):
    """Sums of large terms that cancel to small scores: a plain fp32 sum would
    order many pages differently."""
    b = pu.Batch([1, 1], [6000, 3000], 8, 1, 128, 16, BF, seed=24)
    mn, mx = _bounds(b, 25)
    mid = ((mn.float() + mx.float()) * 500).to(BF)
    # columns in pairs of opposite sign under the same query value
    b.q[..., 1::2] = b.q[..., 0::2]
    mid[..., 1::2] = -mid[..., 0::2]
    noise = (torch.rand_like(mid.float()) * 0.01).to(BF)
    mid = torch.where(mid.abs() < 0.01, noise, mid)
    _check_select(ts, b, 40, 1, 1, mid, mid)


def test_select_scores_that_are_not_finite_rank_last(ts):
    b = pu.Batch([1], [1600], 4, 1, 64, 16, BF, seed=26)
    mn, mx = _bounds(b, 27)
    for i, x in ((3, float("nan")), (17, float("inf")), (40, float("-inf"))):
        (mn if i == 40 else mx)[int(b.table_host[0, i]), 0, 5] = x
    pages, _ = _check_select(ts, b, 30, 1, 1, mn, mx)
    assert not {3, 17, 40} & set(pages[0, 0].tolist())
    # chosen only when nothing better is left, lowest first
    _check_select(ts, b, 96, 1, 1, mn, mx)


def test_select_many_pages(ts):
    """More candidates than one trip of the selection, ragged against it."""
    b = pu.Batch([1, 2], [16 * 5003 + 5, 16 * 513], 2, 1, 64, 16, FP, seed=28)
    mn, mx = _bounds(b, 29)
    for top in (1, 511, 4000):
        _check_select(ts, b, top, 1, 1, mn, mx)


# ------------------------------------------------------------------ attention over chosen pages
def _chosen(b, counts_of, seed=0):
    rng = np.random.default_rng(seed)
    rows = po.token_rows(b.cu, b.kv_lens)
    N = max(counts_of) if counts_of else 1
    pages = np.full((b.n, b.Hkv, N), 2 ** 29, dtype=np.int32)     # wild behind the count
    counts = np.full((b.n, b.Hkv), 0, dtype=np.int32)
    for t, s, p in rows:
        for h in range(b.Hkv):
            vis = p // b.ps + 1
            m = min(vis, counts_of[int(rng.integers(len(counts_of)))])
            pages[t, h, :m] = np.sort(rng.permutation(vis)[:m])
            counts[t, h] = m
    return pages, counts


@pytest.mark.parametrize("dtype", [BF, FP], ids=["bf16", "fp16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("ps", [16, 32, 64, 128])
def test_selected(ts, dtype, d, ps):
    b = pu.Batch([1, 2, 0, 5], [1, 900, 10, 1700], 8, 2, d, ps, dtype, seed=30 + ps, extra=1)
    pages, counts = _chosen(b, [0, 1, 3, 7, 12], seed=ps)
    for t in range(b.n):                       # the list may come in any order
        for h in range(b.Hkv):
            pages[t, h, :counts[t, h]] = np.random.default_rng(t).permutation(pages[t, h, :counts[t, h]])
    o = torch.full_like(b.q, 55.0)
    lse = torch.full((b.n, 8), 55.0, device="cuda")
    ts.ts_paged_attention_selected(b.q, b.k, b.v, b.cu_q, b.lens, b.table,
                                   torch.from_numpy(pages).cuda(), torch.from_numpy(counts).cuda(),
                                   o=o, lse=lse, status=b.status)
    assert status_of(b) == 0
    assert (o[b.cu[-1]:] == 55.0).all() and (lse[b.cu[-1]:] == 55.0).all()
    pu.check_attention(o, lse, b.oracle(pages, counts), dtype, d)


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (8, 8), (40, 8), (16, 1), (20, 1)])
def test_selected_head_groups(ts, Hq, Hkv):
    b = pu.Batch([1, 1, 3], [2000, 77, 640], Hq, Hkv, 128, 16, BF, seed=Hq)
    pages, counts = _chosen(b, [40, 90], seed=Hq)
    o, lse = ts.ts_paged_attention_selected(b.q, b.k, b.v, b.cu_q, b.lens, b.table,
                                            torch.from_numpy(pages).cuda(),
                                            torch.from_numpy(counts).cuda(), status=b.status)
    assert status_of(b) == 0
    pu.check_attention(o, lse, b.oracle(pages, counts), BF, 128)


def test_selected_reports_bad_lists(ts):
    b = pu.Batch([1, 1], [200, 200], 4, 1, 64, 16, BF, seed=31)
    pages, counts = _chosen(b, [6], seed=1)
    for at, x in ((2, -1), (2, 13), (2, 2 ** 29)):
        p = pages.copy()
        p[0, 0, at] = x
        b.status.zero_()
        o, lse = ts.ts_paged_attention_selected(b.q, b.k, b.v, b.cu_q, b.lens, b.table,
                                                torch.from_numpy(p).cuda(),
                                                torch.from_numpy(counts).cuda(), status=b.status)
        assert status_of(b) == 1
        # the listed pages that are right still count
        keep = p.copy()
        keep[0, 0, at] = p[0, 0, 0]
        pu.check_attention(o, lse, b.oracle(keep, counts), BF, 64)
    for x in (-3, 100):
        c = counts.copy()
        c[0, 0] = x
        b.status.zero_()
        ts.ts_paged_attention_selected(b.q, b.k, b.v, b.cu_q, b.lens, b.table,
                                       torch.from_numpy(pages).cuda(), torch.from_numpy(c).cuda(),
                                       status=b.status)
        assert status_of(b) == 1


# ------------------------------------------------------------------ together
@pytest.mark.parametrize("dtype", [BF, FP], ids=["bf16", "fp16"])
def test_prompt_in_chunks_then_sparse_decoding(ts, dtype):
    """A prompt enters in chunks and decoding goes on over chosen pages, every
    operator fed by the one before it; each stage is checked on the values it
    was given.  With every page chosen, the sparse form gives the dense one."""
    Hq, Hkv, d, ps = 32, 2, 128, 16
    total = 700
    b = pu.Batch([0], [total], Hq, Hkv, d, ps, dtype, seed=40)
    b.k.fill_(float("nan"))
    b.v.fill_(float("nan"))
    mn, mx = (torch.full((b.n_pages, Hkv, d), float("nan"), dtype=dtype, device="cuda")
              for _ in range(2))
    freqs, scale = ts.ts_rope_frequencies(d, scaling="linear", factor=2.0)
    done = 0
    for new in (300, 1, 250, 100, 1, 1):
        b.q_lens, b.cu, b.n = [new], [0, new], new
        b.cu_q = torch.tensor([0, new], dtype=torch.int32, device="cuda")
        done += new
        b.kv_lens = [done]
        b.lens = torch.tensor([done], dtype=torch.int32, device="cuda")
        q, k, v = (torch.randn(new, h, d, device="cuda").to(dtype) for h in (Hq, Hkv, Hkv))
        b.q = ts.ts_paged_rope_append(q, k, v, b.cu_q, b.lens, b.table, b.k, b.v, freqs,
                                      rope_scale=scale, key_min=mn, key_max=mx, status=b.status)
        o, lse = _check_attend(ts, b)
        pages, counts = _check_select(ts, b, 6, 1, 2, mn, mx)
        os_, ls = ts.ts_paged_attention_selected(b.q, b.k, b.v, b.cu_q, b.lens, b.table, pages,
                                                 counts, status=b.status)
        assert status_of(b) == 0
        pu.check_attention(os_, ls, b.oracle(pages.cpu().numpy(), counts.cpu().numpy()), dtype, d)
        # the pages' bounds hold every key
        rows = b.k[b.table_host[0, :(done + ps - 1) // ps].long()].float()
        lo, hi = (x[b.table_host[0, :(done + ps - 1) // ps].long()].float()[:, :, None]
                  for x in (mn, mx))
        seen = ~torch.isnan(rows)
        assert ((rows >= lo) | ~seen).all() and ((rows <= hi) | ~seen).all()
        pages, counts = _check_select(ts, b, 60, 1, 2, mn, mx)
        os_, ls = ts.ts_paged_attention_selected(b.q, b.k, b.v, b.cu_q, b.lens, b.table, pages,
                                                 counts)
        pu.check_attention(os_, ls, b.oracle(), dtype, d)


def test_matches_verification_of_a_chain(ts):
    """A chain of draft tokens verified over a contiguous cache and the same
    rows as a chunk over pages: one definition, two kernels."""
    Hq, Hkv, d, ps, T, L = 16, 4, 128, 32, 12, 500
    b = pu.Batch([T], [L + T], Hq, Hkv, d, ps, BF, seed=41)
    ids = b.table_host[0, :(L + T + ps - 1) // ps].long()
    flat = lambda x: x[ids].permute(1, 0, 2, 3).reshape(Hkv, -1, d)[:, :L + T].contiguous()  # noqa: E731
    parents = torch.arange(-1, T - 1, dtype=torch.int32, device="cuda")
    o1, lse1, _ = ts.ts_verify_attention(b.q, flat(b.k), flat(b.v), L, parents, want_imp=False,
                                         status=b.status)
    o2, lse2 = _check_attend(ts, b)
    assert torch.allclose(lse1, lse2, rtol=0, atol=1e-4)
    # verification rounds P to fp16 and its partial rows to fp16 (2^-11 each)
    bound = 2.0 ** -8 * o1.abs() + 2.0 ** -7
    assert ((o1 - o2.float()).abs() <= bound).all()
