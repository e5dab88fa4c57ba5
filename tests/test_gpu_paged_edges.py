"""GPU: the paged calls where their numbers and their paths go to the edge:
attention sinks, weights of few keys, queries that are not finite, channels far
apart in size, tables that are wrong where no token looks, long candidate lists,
plans of many short tiles, and calls on a stream of their own."""
import numpy as np
import pytest
import torch

from oracle import paged_oracle as po
import paged_util as pu

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def ts():
    import self_speculative_ultra_gb300 as ts
    ts.build()
    return ts


# ------------------------------------------------------------------ attention sinks
class Stream:
    """One stream whose rows lie in shuffled pages; k, v [Hkv, kv, d]."""

    def __init__(self, q, k, v, ps):
        Hkv, kv, d = k.shape
        self.q, self.n, self.Hq, self.Hkv, self.d, self.kv, self.ps = \
            q, q.shape[0], q.shape[1], Hkv, d, kv, ps
        m = (kv + ps - 1) // ps
        perm = torch.randperm(m, generator=torch.Generator().manual_seed(1)).cuda()
        self.table = perm.int()[None].contiguous()
        self.rows = (k, v)

        def pool(x):
            pages = torch.zeros(m, Hkv, ps, d, dtype=x.dtype, device="cuda")
            pad = torch.cat([x, x.new_zeros(Hkv, m * ps - kv, d)], 1)
            pages[perm] = pad.view(Hkv, m, ps, d).permute(1, 0, 2, 3)
            return pages
        self.k, self.v = pool(k), pool(v)
        self.cu_q = torch.tensor([0, self.n], dtype=torch.int32, device="cuda")
        self.lens = torch.tensor([kv], dtype=torch.int32, device="cuda")
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def reference(self):
        """(o, lse, sum p |v|, largest sum |q k| / sqrt d) in 64 bits."""
        G, n = self.Hq // self.Hkv, self.n
        last = torch.arange(self.kv - n, self.kv, device="cuda")
        hide = torch.arange(self.kv, device="cuda")[None, None] > last[:, None, None]
        out = []
        for h in range(self.Hkv):
            q = self.q[:, h * G:(h + 1) * G].double()
            k, v = (x[h].double() for x in self.rows)
            x = (q @ k.t() / self.d ** 0.5).masked_fill(hide, -float("inf"))
            lse = x.logsumexp(2)
            p = (x - lse[..., None]).exp()
            aq = (q.abs() @ k.abs().t()).masked_fill(hide, 0.0).amax(2) / self.d ** 0.5
            out.append((p @ v, lse, p @ v.abs(), aq))
        return tuple(torch.cat(x, 1).cpu().numpy() for x in zip(*out))


def _sink_stream(q, kv, Hq, Hkv, d, ps, dtype, nats, at, seed):
    """Row `at` stands `nats` above all others and has a value of zero, so the
    outputs are the tail's alone.  The others' scores spread by a quarter nat."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    qs, k, v = rnd(q, Hq, d) * 0.5, rnd(Hkv, kv, d) * 0.5, 1.0 + 0.25 * rnd(Hkv, kv, d)
    qs[..., 0] = 8.0
    k[..., 0] = 0.0
    k[:, at] = 0.0
    k[:, at, 0] = nats * d ** 0.5 / 8.0
    v[:, at] = 0.0
    return Stream(qs.to(dtype), k.to(dtype), v.to(dtype), ps)


def _check_sink(o, lse, ref, dtype, d, p_round):
    """check_attention's bound, and what a 16-bit weight may lose beside a key far
    above it in the same 128 keys: for fp16 at most 2^-32 of the largest there a
    weight, 2^-25 a tile, times the largest |v| (below 4 here)."""
    O, L, av, aq = ref
    e_w = 3 * d * 2.0 ** -23 * aq + 2.0 ** -20
    delta = (2 * e_w + p_round + 2.0 ** -18)[..., None] * av
    if dtype == FP:
        delta = delta + 4 * 2.0 ** -25
    err = np.abs(pu.f64(o) - O) - (pu.U[dtype] * (np.abs(O) + delta) + delta + pu.TINY[dtype])
    assert err.max() <= 0, f"o off by {err.max():.3e} beyond its bound, |o| {np.abs(O).mean():.3e}"
    el = np.abs(pu.f64(lse) - L) - (2 * e_w + 2.0 ** -22 * np.abs(L))
    assert el.max() <= 0


SINKS = [(FP, 16.0), (FP, 17.0), (FP, 18.0), (FP, 20.0), (FP, 24.0), (FP, 60.0), (BF, 18.0)]
SINK_IDS = [f"{'fp16' if t is FP else 'bf16'}-{x:g}" for t, x in SINKS]


@pytest.mark.parametrize("dtype,nats", SINKS, ids=SINK_IDS)
@pytest.mark.parametrize("at", [0, 20001])
@pytest.mark.parametrize("q,kv,Hq,Hkv,d", [(1, 102400, 8, 2, 128),   # units cut in stretches
                                           (1, 30000, 4, 1, 64),     # a cluster a unit
                                           (3, 60000, 12, 2, 64)])
def test_tail_behind_a_sink_few_rows(ts, q, kv, Hq, Hkv, d, at, dtype, nats):
    s = _sink_stream(q, kv, Hq, Hkv, d, 64, dtype, nats, at, 3)
    o, lse = ts.ts_paged_attention(s.q, s.k, s.v, s.cu_q, s.lens, s.table, q, status=s.status)
    assert int(s.status.item()) == 0
    # a weight is a 16-bit value and its remainder: off by 2^-16 (bf16); fp16: 2^-22,
    # and where it is small 2^-25 of a step in which its 32 keys' largest is 2^8 or more
    _check_sink(o, lse, s.reference(), dtype, d, 2.0 ** -16)


@pytest.mark.parametrize("dtype,nats", SINKS, ids=SINK_IDS)
@pytest.mark.parametrize("at", [0, 20001])
def test_tail_behind_a_sink_chosen_pages(ts, at, dtype, nats):
    s = _sink_stream(1, 40000, 8, 2, 128, 32, dtype, nats, at, 4)
    m = s.table.shape[1]
    pages = torch.arange(m, dtype=torch.int32, device="cuda").expand(1, 2, m).contiguous()
    counts = torch.full((1, 2), m, dtype=torch.int32, device="cuda")
    o, lse = ts.ts_paged_attention_selected(s.q, s.k, s.v, s.cu_q, s.lens, s.table, pages, counts,
                                            status=s.status)
    assert int(s.status.item()) == 0
    _check_sink(o, lse, s.reference(), dtype, 128, 2.0 ** -16)


@pytest.mark.parametrize("dtype,nats", SINKS, ids=SINK_IDS)
@pytest.mark.parametrize("at", [0, 20001])
@pytest.mark.parametrize("d", [64, 128])
def test_tail_behind_a_sink_tiles(ts, d, at, dtype, nats):
    s = _sink_stream(90, 40000, 4, 1, d, 64, dtype, nats, at, 5)
    o, lse = ts.ts_paged_attention(s.q, s.k, s.v, s.cu_q, s.lens, s.table, 90, status=s.status)
    assert int(s.status.item()) == 0
    # one 16-bit value: half a step a weight; fp16: a row whose weights sum to 2^-7
    # or more over 128 keys has lost at most 128 * 2^-25 = 2^-11 of the sum besides
    _check_sink(o, lse, s.reference(), dtype, d, 2.0 ** -8 if dtype == BF else 2.0 ** -10)


@pytest.mark.parametrize("q,Hq", [(1, 4), (90, 4)])
@pytest.mark.parametrize("dtype", [BF, FP], ids=["bf16", "fp16"])
def test_scores_that_swing_from_tile_to_tile(ts, q, Hq, dtype):
    """Stretches of keys up and down by tens of nats, both ways: the reference of
    the weights follows within its bounds."""
    g = torch.Generator(device="cuda").manual_seed(6)
    kv, d = 40000, 64
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    qs, k, v = rnd(q, Hq, d) * 0.5, rnd(1, kv, d) * 0.5, rnd(1, kv, d)
    qs[..., 0] = 8.0
    level = torch.randint(-60, 61, ((kv + 99) // 100,), generator=g, device="cuda").float()
    k[0, :, 0] = level.repeat_interleave(100)[:kv]
    s = Stream(qs.to(dtype), k.to(dtype), v.to(dtype), 64)
    o, lse = ts.ts_paged_attention(s.q, s.k, s.v, s.cu_q, s.lens, s.table, q, status=s.status)
    assert int(s.status.item()) == 0
    _check_sink(o, lse, s.reference(), dtype, d, 2.0 ** -8 if dtype == BF else 2.0 ** -10)


@pytest.mark.parametrize("dtype", [BF, FP], ids=["bf16", "fp16"])
@pytest.mark.parametrize("Hq", [1, 16])
def test_few_rows_keep_the_remainder_of_a_weight(ts, dtype, Hq):
    """Eight keys whose values cancel in pairs: the outputs are far below sum p|v|,
    so a weight of one 16-bit value (2^-9, 2^-12 on average) would show."""
    g = torch.Generator(device="cuda").manual_seed(7)
    d = 128
    k = torch.randn(1, 8, d, generator=g, device="cuda")
    k[:, 1::2] = k[:, 0::2]
    k[:, 1::2] += 0.03 * torch.randn(1, 4, d, generator=g, device="cuda")
    v = torch.randn(1, 8, d, generator=g, device="cuda")
    v[:, 1::2] = -v[:, 0::2]
    q = torch.randn(1, Hq, d, generator=g, device="cuda") * 0.02
    s = Stream(q.to(dtype), k.to(dtype), v.to(dtype), 16)
    o, lse = ts.ts_paged_attention(s.q, s.k, s.v, s.cu_q, s.lens, s.table, 1, status=s.status)
    assert int(s.status.item()) == 0
    ref = s.reference()
    # half a step of either part's rounding, relative: bf16 2^-16, fp16 2^-22
    pu.check_attention(o, lse, ref, dtype, d, p_round=2.0 ** -16 if dtype == BF else 2.0 ** -22)
    # the case shows it: with the weights rounded once the bound is broken
    x = s.q[0].double() @ s.rows[0][0].double().t() / d ** 0.5
    p = (x - x.amax(1, keepdim=True)).exp()
    once = (p.to(dtype).double() @ s.rows[1][0].double() / p.sum(1, keepdim=True)).to(dtype)
    with pytest.raises(AssertionError):
        pu.check_attention(once[None], lse, ref, dtype, d,
                           p_round=2.0 ** -16 if dtype == BF else 2.0 ** -22)


# ------------------------------------------------------------------ choice of pages
class Bounds:
    """A batch for the choice alone: tables and bounds, no rows."""

    def __init__(self, q_lens, kv_lens, Hq, Hkv, d, ps, dtype, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")
        self.cu = [0]
        for x in q_lens:
            self.cu.append(self.cu[-1] + x)
        self.kv_lens, self.n, self.Hkv, self.d, self.ps = kv_lens, self.cu[-1], Hkv, d, ps
        need = [(x + ps - 1) // ps for x in kv_lens]
        self.n_pages = sum(need)
        perm = torch.randperm(self.n_pages, generator=torch.Generator().manual_seed(seed)).int()
        table = torch.zeros(len(need), max(need), dtype=torch.int32)
        at = 0
        for s, m in enumerate(need):
            table[s, :m] = perm[at:at + m]
            at += m
        self.table_host, self.table = table, table.cuda()
        self.q = self.rnd(self.n, Hq, d).to(dtype)
        mid, half = self.rnd(self.n_pages, Hkv, d), self.rnd(self.n_pages, Hkv, d).abs()
        self.mn, self.mx = (mid - half).to(dtype), (mid + half).to(dtype)
        self.cu_q = torch.tensor(self.cu, dtype=torch.int32, device="cuda")
        self.lens = torch.tensor(kv_lens, dtype=torch.int32, device="cuda")
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def check(self, ts, n_top, n_sink, n_recent):
        pages, counts = ts.ts_paged_select_pages(self.q, self.mn, self.mx, self.cu_q, self.lens,
                                                 self.table, self.ps, n_top, n_sink, n_recent,
                                                 status=self.status)
        assert int(self.status.item()) == 0
        P, C = po.select_pages(pu.f64(self.q), pu.f64(self.mn), pu.f64(self.mx), self.cu,
                               self.kv_lens, self.table_host.numpy(), self.ps, n_top, n_sink,
                               n_recent)
        np.testing.assert_array_equal(counts.cpu().numpy(), C)
        np.testing.assert_array_equal(pages.cpu().numpy(), P)


@pytest.mark.parametrize("dtype", [BF, FP], ids=["bf16", "fp16"])
@pytest.mark.parametrize("Hq", [1, 4])
@pytest.mark.parametrize("what", [float("nan"), float("inf"), -float("inf")])
def test_choice_with_a_query_that_is_not_finite(ts, dtype, Hq, what):
    """No score of that token and KV head is finite: all pages rank last, the
    lowest are taken.  The other tokens choose as ever."""
    b = Bounds([1, 2], [3000, 5000], 2 * Hq, 2, 64, 16, dtype, seed=8)
    b.q[1, Hq, 9] = what
    with np.errstate(invalid="ignore"):
        b.check(ts, 20, 1, 2)
        b.check(ts, 100, 0, 1)


@pytest.mark.parametrize("dtype", [BF, FP], ids=["bf16", "fp16"])
@pytest.mark.parametrize("big", [1.0, 2048.0, 32768.0])
def test_choice_beside_a_large_query_channel_without_keys(ts, dtype, big):
    """A channel of large queries and zero keys: the scores are the small channels'
    alone, to their last bits."""
    b = Bounds([1, 1], [90000, 40000], 2, 1, 64, 16, dtype, seed=9)
    b.q = (b.rnd(2, 2, 64) * 2.0 ** -13).to(dtype)
    b.q[..., 5] = big
    b.mn[..., 5] = b.mx[..., 5] = 0.0
    for top in (50, 700, 2000):
        b.check(ts, top, 1, 1)


@pytest.mark.parametrize("coarse", [None, 1.0, 0.0])
def test_choice_among_more_pages_than_shared_memory_holds(ts, coarse):
    """50,000 candidates: scores apart (all near the cut fit, or few are ranked) and
    scores that tie in their thousands (all are ranked again)."""
    b = Bounds([1, 2], [16 * 50100, 16 * 49160], 2, 1, 64, 16, BF, seed=10)
    if coarse is not None:
        b.q = (b.q * 2).round()
        b.mn, b.mx = (x.float().mul(coarse).round().to(BF) for x in (b.mn, b.mx))
    for top in (1, 700, 49000):
        b.check(ts, top, 1, 1)
    if coarse is None:
        # neighbours at the cut that only well formed scores rank
        b.mx = b.mx[:1].expand_as(b.mx).clone()
        b.mn = b.mn[:1].expand_as(b.mn).clone()
        pick = torch.arange(0, b.n_pages, 997, device="cuda")
        bits = b.mx.view(torch.int16)
        bits[pick, 0, (pick // 997) % 64] = bits[pick, 0, (pick // 997) % 64] + 1
        for top in (20, 80):
            b.check(ts, top, 1, 1)


@pytest.mark.parametrize("cu,lens", [([0, 1, 1, 2], [900, 10 ** 9, 700]),   # no token of its own
                                     ([0, 1, 1, 2], [900, -1, 700]),
                                     ([0, 2, 1, 2], [900, 500, 700]),      # falls behind a token
                                     ([0, 1, 2, 9], [900, 500, 700])])
def test_every_call_reports_a_bad_batch(ts, cu, lens):
    b = Bounds([1, 1, 0], [900, 500, 700], 4, 2, 64, 16, BF, seed=11)
    cu_q = torch.tensor(cu, dtype=torch.int32, device="cuda")
    ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
    kp = torch.zeros(b.n_pages, 2, 16, 64, dtype=BF, device="cuda")
    vp, x = torch.zeros_like(kp), torch.zeros(2, 2, 64, dtype=BF, device="cuda")
    freqs, _ = ts.ts_rope_frequencies(64)
    pages = torch.zeros(2, 2, 1, dtype=torch.int32, device="cuda")
    counts = torch.ones(2, 2, dtype=torch.int32, device="cuda")
    calls = [lambda st: ts.ts_paged_select_pages(b.q, b.mn, b.mx, cu_q, ln, b.table, 16, 8, 1, 1, status=st),
             lambda st: ts.ts_paged_select_pages(b.q, b.mn, b.mx, cu_q, ln, b.table, 16, 900, 1, 1, status=st),
             lambda st: ts.ts_paged_attention(b.q, kp, vp, cu_q, ln, b.table, 2, status=st),
             lambda st: ts.ts_paged_attention_selected(b.q, kp, vp, cu_q, ln, b.table, pages, counts, status=st),
             lambda st: ts.ts_paged_rope_append(b.q, x, x, cu_q, ln, b.table, kp, vp, freqs, status=st)]
    for i, call in enumerate(calls):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        call(status)
        assert int(status.item()) == 1, i


# ------------------------------------------------------------------ plans, waits, streams
@pytest.mark.parametrize("Hkv,long", [(1, 0), (1, 3000), (2, 3000)])
def test_thousands_of_short_tiles(ts, Hkv, long):
    """More sequences than the plan's threads and more tiles than its shared memory
    holds; with few KV heads some may be cut."""
    rng = np.random.default_rng(12)
    n_seq, Hq, d, ps = 2300, 8 * Hkv, 64, 16
    ql = rng.integers(0, 10, n_seq)
    kl = np.maximum(ql, rng.integers(0, 60, n_seq))
    ql[5], kl[5] = 9, 57
    if long:
        kl[7] = kl[1500] = kl[2200] = long
    b = pu.Batch([int(x) for x in ql], [int(x) for x in kl], Hq, Hkv, d, ps, BF, seed=13, extra=2)
    o = torch.full((b.n, Hq, d), 55.0, dtype=BF, device="cuda")
    lse = torch.full((b.n, Hq), 55.0, device="cuda")
    ts.ts_paged_attention(b.q, b.k, b.v, b.cu_q, b.lens, b.table, 9, o=o, lse=lse, status=b.status)
    assert int(b.status.item()) == 0
    assert (o[b.cu[-1]:] == 55.0).all() and (lse[b.cu[-1]:] == 55.0).all()
    pu.check_attention(o, lse, b.oracle(), BF, d, p_round=2.0 ** -8)


@pytest.mark.parametrize("d", [64, 128])
def test_expired_wait_of_the_chunk_kernel_is_reported(ts, d):
    """With a limit of one clock a wait that outlasts one hardware attempt is given
    up, reported, and the kernel returns.  Items of a hundred microseconds have such
    waits (for the next item, for the place of its queries); the call behind it is
    right."""
    g = torch.Generator(device="cuda").manual_seed(16)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").to(BF)  # noqa: E731
    s = Stream(rnd(200, 32, d), rnd(2, 60000, d), rnd(2, 60000, d), 32)
    ts.ts_set_wait_limit(1)
    try:
        ts.ts_paged_attention(s.q, s.k, s.v, s.cu_q, s.lens, s.table, 200, status=s.status)
        torch.cuda.synchronize()
    finally:
        ts.ts_set_wait_limit(0)
    assert int(s.status.item()) == 4
    s.status.zero_()
    o, lse = ts.ts_paged_attention(s.q, s.k, s.v, s.cu_q, s.lens, s.table, 200, status=s.status)
    assert int(s.status.item()) == 0
    pu.check_attention(o, lse, s.reference(), BF, d, p_round=2.0 ** -8)


@pytest.mark.parametrize("which", ["append", "attend", "tiles", "select", "selected"])
def test_a_call_on_its_own_stream_leaves_freed_memory_to_its_readers(ts, which):
    """Memory freed on the current stream while kernels queued there still read it
    must not become an output or the workspace of a call on another stream."""
    q = 200 if which == "tiles" else 2
    b = pu.Batch([q] * 3, [3000, 2100, 800], 32, 2, 128, 32, BF, seed=14)
    x = torch.randn(b.n, 2, 128, device="cuda").to(BF)
    freqs, _ = ts.ts_rope_frequencies(128)
    mn, mx = b.k.nan_to_num().amin(2), b.k.nan_to_num().amax(2)
    pages = torch.zeros(b.n, 2, 4, dtype=torch.int32, device="cuda")
    pages[:] = torch.arange(4, dtype=torch.int32, device="cuda")
    counts = torch.full((b.n, 2), 4, dtype=torch.int32, device="cuda")

    def call(stream):
        if which == "append":
            return [ts.ts_paged_rope_append(b.q, x, x, b.cu_q, b.lens, b.table, b.k, b.v, freqs,
                                            stream=stream)]
        if which == "select":
            return list(ts.ts_paged_select_pages(b.q, mn, mx, b.cu_q, b.lens, b.table, 32, 8, 1, 1,
                                                 stream=stream))
        if which == "selected":
            return list(ts.ts_paged_attention_selected(b.q, b.k, b.v, b.cu_q, b.lens, b.table,
                                                       pages, counts, stream=stream))
        return list(ts.ts_paged_attention(b.q, b.k, b.v, b.cu_q, b.lens, b.table, q, stream=stream))
    want = call(None)
    sizes = sorted({t.untyped_storage().nbytes() for t in want} |
                   {ts.ts_paged_attention_workspace_bytes(b.n, 3, 32, 2, 128, b.table.shape[1], 32, q),
                    ts.ts_paged_select_workspace_bytes(b.n, 2, b.table.shape[1])})
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    busy = [torch.full((s,), 91, dtype=torch.uint8, device="cuda") for s in sizes if s for _ in range(40)]
    kept = [torch.zeros_like(t) for t in busy]
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)              # a tenth of a second
    for k, t in zip(kept, busy):
        k.copy_(t)                              # queued readers
    del busy, t
    got = call(st)
    torch.cuda.synchronize()
    for k in kept:
        assert (k == 91).all()
    for a, c in zip(got, want):
        assert torch.equal(a, c)


def test_outputs_of_a_call_on_its_own_stream_outlive_their_readers(ts):
    """An output that a queued kernel of the current stream still reads is not
    handed out again on the call's stream once it is freed."""
    b = pu.Batch([2] * 3, [3000, 2100, 800], 32, 2, 128, 32, BF, seed=15)
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    o = ts.ts_paged_attention(b.q, b.k, b.v, b.cu_q, b.lens, b.table, 2, stream=st)[0]
    st.synchronize()
    want, kept = o.clone(), torch.zeros_like(o)
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)
    kept.copy_(o)
    del o
    with torch.cuda.stream(st):
        others = [torch.full_like(want, 5.0) for _ in range(8)]
    torch.cuda.synchronize()
    assert torch.equal(kept, want) and len(others) == 8


@pytest.mark.parametrize("own", [False, True], ids=["current", "own-stream"])
@pytest.mark.parametrize("dtype", [BF, FP], ids=["bf16", "fp16"])
def test_a_captured_step_replayed_on_new_tokens(ts, dtype, own):
    """Append, choice, and both attentions in one graph, on the capture's stream or
    forked to another: replays on new queries, lengths and tables give what eager calls
    give, and two replays of a step end in the same bits."""
    b = pu.Batch([3, 1, 0, 2], [2100, 900, 40, 1700], 8, 2, 128, 16, dtype, seed=17, extra=2)
    b.k.nan_to_num_(nan=0.0)
    b.v.nan_to_num_(nan=0.0)
    mn, mx = b.k.amin(2).contiguous(), b.k.amax(2).contiguous()
    pools = (b.k, b.v, mn, mx)
    freqs, _ = ts.ts_rope_frequencies(128)
    g = torch.Generator(device="cuda").manual_seed(18)
    fresh = lambda h: torch.randn(b.n, h, 128, generator=g, device="cuda").to(dtype)  # noqa: E731
    q, k, v = fresh(8), fresh(2), fresh(2)

    def step(stream=None):
        kw = dict(status=b.status, stream=stream)
        r = ts.ts_paged_rope_append(q, k, v, b.cu_q, b.lens, b.table, b.k, b.v, freqs,
                                    key_min=mn, key_max=mx, **kw)
        pages, counts = ts.ts_paged_select_pages(r, mn, mx, b.cu_q, b.lens, b.table, 16, 9, 1, 2, **kw)
        sparse = ts.ts_paged_attention_selected(r, b.k, b.v, b.cu_q, b.lens, b.table, pages, counts, **kw)
        dense = ts.ts_paged_attention(r, b.k, b.v, b.cu_q, b.lens, b.table, 3, **kw)
        return (r, pages, counts) + sparse + dense
    side = torch.cuda.Stream()
    warm = torch.cuda.Stream()
    with torch.cuda.stream(warm):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        if own:
            side.wait_stream(torch.cuda.current_stream())
        outs = step(side if own else None)
        if own:
            torch.cuda.current_stream().wait_stream(side)
    live = b.cu[-1]
    for lens in ([2100, 900, 40, 1700], [2050, 17, 40, 3], [3, 1, 0, 2]):
        b.lens.copy_(torch.tensor(lens, dtype=torch.int32))
        for x, h in ((q, 8), (k, 2), (v, 2)):
            x.copy_(fresh(h))
        start = [x.clone() for x in pools]
        want = [x[:live].clone() for x in step()]
        pool_want = [x.clone() for x in pools]
        for _ in range(2):
            for x, y in zip(pools, start):
                x.copy_(y)
            graph.replay()
            torch.cuda.synchronize()
            assert int(b.status.item()) == 0
            for x, y in zip(outs, want):
                assert torch.equal(x[:live], y)
            for x, y in zip(pools, pool_want):
                assert torch.equal(x, y)


def test_choices_and_reads_on_two_streams_at_once(ts):
    """The sparse step on two streams, each with its own memory, while both run."""
    bs = [pu.Batch([1, 2, 1], [9000, 5000, 7000], 8, 2, 128, 16, FP, seed=s) for s in (51, 52)]
    bounds = [tuple(f(b.k.nan_to_num(nan=0.0), 2).contiguous() for f in (torch.amin, torch.amax)) for b in bs]

    def step(b, mm, stream=None):
        pages, counts = ts.ts_paged_select_pages(b.q, *mm, b.cu_q, b.lens, b.table, 16, 50, 1, 2,
                                                 stream=stream)
        return (pages, counts) + ts.ts_paged_attention_selected(b.q, b.k, b.v, b.cu_q, b.lens, b.table,
                                                                pages, counts, stream=stream)
    want = [step(b, mm) for b, mm in zip(bs, bounds)]
    streams = [torch.cuda.Stream() for _ in bs]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(8):
        for i in range(2):
            got[i].append(step(bs[i], bounds[i], streams[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for out in got[i]:
            for x, y in zip(out, want[i]):
                assert torch.equal(x, y)
