"""GPU parity of the logits' biases, penalties and masks and of the token counts
they read, and a run of them with the draft trees over a paged cache."""
import numpy as np
import pytest
import torch

from oracle import logits_oracle as lo
from oracle import paged_oracle as po
from oracle import ts_oracle as orc
import paged_util as pu
from test_gpu_paged_tree import parents_of

pytestmark = pytest.mark.gpu
BF, FP, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def ts():
    import self_speculative_ultra_gb300 as ts
    ts.build()
    return ts


def cuda(x, dtype=None):
    return torch.as_tensor(np.ascontiguousarray(x)).to(dtype).cuda() if dtype else \
        torch.as_tensor(np.ascontiguousarray(x)).cuda()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Case:
    """A batch of rows; tokens behind the last sequence, biases, masks and a state."""

    def __init__(self, q_lens, V, dtype, seed=0, extra=0, pad=0, tree=True, n_bias=0, masks="none",
                 counts=True, history=None):
        rng = np.random.default_rng(seed)
        self.q_lens, self.V, self.n_seq, self.rng = q_lens, V, len(q_lens), rng
        self.cu = [0]
        for x in q_lens:
            self.cu.append(self.cu[-1] + x)
        self.n = n = self.cu[-1] + extra
        ns = self.n_seq
        full = torch.from_numpy(rng.standard_normal((max(n, 1), V + pad)) * 3).to(dtype).cuda()
        self.logits = full[:n, :V]
        self.seen = rng.random((ns, V)) < 0.3
        self.counts = (rng.integers(0, 4, (ns, V)) * self.seen).astype(np.int32)
        self.has_counts = counts
        self.rep, self.freq, self.pres = (rng.uniform(*r, ns).astype(np.float32)
                                          for r in ((0.7, 2.0), (-0.5, 1.0), (-0.5, 1.0)))
        self.tree = tree
        self.parents = parents_of(q_lens, "mixed", seed=seed, extra=extra) if tree else None
        self.tokens = rng.integers(0, V, n).astype(np.int32)
        if tree and V > 5:
            self.tokens[::3] = 5                       # a token that paths hold many times
        self.bias_ids = self.bias = None
        if n_bias:
            self.bias_ids = rng.integers(-1, V, (ns, n_bias)).astype(np.int32)
            self.bias = (rng.standard_normal((ns, n_bias)) * 4).astype(np.float32)
        self.mask = self.mask_rows = None
        if masks != "none":
            m = n if masks == "each" else 3
            self.mask = rng.random((m, V)) < 0.3
            self.mask[0] = False                       # nothing allowed
            if masks == "shared":
                self.mask_rows = rng.integers(-1, 3, n).astype(np.int32)
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def args(self):
        kw = dict(seen=cuda(lo.pack(self.seen)), repetition=cuda(self.rep),
                  frequency=cuda(self.freq), presence=cuda(self.pres))
        if self.has_counts:
            kw["counts"] = cuda(self.counts)
        if self.tree:
            kw.update(tree_tokens=cuda(self.tokens), parents=self.parents)
        if self.bias is not None:
            kw.update(bias_ids=cuda(self.bias_ids), bias=cuda(self.bias))
        if self.mask is not None:
            words = lo.pack(self.mask)
            if self.V % 32:                            # bits behind the vocabulary mean nothing
                words[:, -1] |= np.int32(-1) << (self.V % 32)
            kw["mask"] = cuda(words)
        if self.mask_rows is not None:
            kw["mask_rows"] = cuda(self.mask_rows)
        return kw

    def row(self, s, i, literal, masked=-np.inf):
        t = self.cu[s] + i
        path = []
        if self.tree:
            par = self.parents[self.cu[s]:self.cu[s + 1]].tolist()
            path = [int(self.tokens[self.cu[s] + a]) for a in po.root_paths(par)[i][1:]]
        bias = {}
        if self.bias is not None:
            bias = {int(k): float(b) for k, b in zip(self.bias_ids[s], self.bias[s]) if k >= 0}
        allowed = None
        if self.mask is not None:
            r = t if self.mask_rows is None else int(self.mask_rows[t])
            allowed = self.mask[r] if r >= 0 else None
        counts = self.counts[s] if self.has_counts else np.zeros(self.V, dtype=np.int64)
        return lo.process_row(self.logits[t].double().cpu().numpy(), bias, self.seen[s], counts,
                              path, self.rep[s], self.freq[s], self.pres[s], allowed, masked, literal)

    def check(self, out, masked=-np.inf):
        got = out.cpu().numpy()
        for s in range(self.n_seq):
            for i in range(self.q_lens[s]):
                y = got[self.cu[s] + i].astype(np.float64)
                Y, err = self.row(s, i, False, masked)
                fine = np.isfinite(Y)
                np.testing.assert_array_equal(y[~fine], Y[~fine])
                assert (np.abs(y[fine] - Y[fine]) <= err[fine]).all()
                # each operation is rounded once, as the header says: the very bits
                bits, _ = self.row(s, i, True, masked)
                np.testing.assert_array_equal(y.astype(np.float32), bits)

    def run(self, ts, **kw):
        out = torch.full((self.n, self.V), 55.0, device="cuda")
        r = ts.ts_logits_process(self.logits, i32(self.cu), out=out, status=self.status,
                                 **{**self.args(), **kw})
        assert r is out
        torch.cuda.synchronize()
        assert int(self.status.item()) == 0
        assert (out[self.cu[-1]:] == 55.0).all()       # rows behind the last sequence
        self.check(out, kw.get("masked_value", -np.inf))
        return out


@pytest.mark.parametrize("dtype", [F32, BF, FP], ids=["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("V", [1, 31, 32, 33, 1000, 4095, 4096, 4097, 12344, 20003])
def test_everything_at_once(ts, dtype, V):
    Case([7, 0, 1, 40, 64], V, dtype, seed=V, extra=2, n_bias=40, masks="each").run(ts)


@pytest.mark.parametrize("dtype", [F32, BF, FP], ids=["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("pad", [0, 1, 4, 8, 24])
@pytest.mark.parametrize("V", [8192, 5001])
def test_row_strides(ts, dtype, pad, V):
    Case([3, 9], V, dtype, seed=pad, pad=pad, n_bias=9, masks="shared").run(ts)


@pytest.mark.parametrize("dtype", [F32, BF, FP], ids=["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("V", [2, 34, 4098, 20002])
def test_even_vocabularies(ts, dtype, V):
    """Rows on a boundary of two values but not of four."""
    Case([7, 0, 1, 40, 64], V, dtype, seed=V, extra=2, n_bias=40, masks="each").run(ts)


@pytest.mark.parametrize("dtype", [F32, BF, FP], ids=["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("V,pad", [(8192, 2), (8194, 2), (8194, 4), (8194, 1)])
def test_even_row_strides(ts, dtype, V, pad):
    Case([3, 9], V, dtype, seed=pad, pad=pad, n_bias=9, masks="shared").run(ts)


def test_even_rows_in_place(ts):
    for V, pad in ((4098, 4), (8192, 2)):
        c = Case([9, 30], V, F32, seed=4, n_bias=5, masks="each", pad=pad)
        want = c.run(ts)
        r = ts.ts_logits_process(c.logits, i32(c.cu), out=c.logits, **c.args())
        assert r is c.logits and torch.equal(r, want)


@pytest.mark.parametrize("dtype", [F32, BF, FP], ids=["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("V", [20001, 20002, 20004])
def test_runs_of_rows(ts, dtype, V):
    """8 or 9 rows a block: runs that begin inside trees and go from one to the next,
    whose paths hold a token many times, a mask a row; single rows and streams without
    a node among them."""
    q = [64, 40, 57, 1, 0, 64, 1, 1, 63, 48, 64, 51, 64, 3, 64, 60, 64, 64]
    c = Case(q, V, dtype, seed=V, extra=7, n_bias=60, masks="each")
    c.tokens[1::3] = c.rng.integers(0, 40, c.tokens[1::3].shape)
    # 152 SMs hold 6 blocks of 2048 values each
    assert c.n * ((V + 2047) // 2048) // (152 * 6) in (8, 9)
    out = torch.full((c.n, V), 55.0, device="cuda")
    ts.ts_logits_process(c.logits, i32(c.cu), out=out, status=c.status, **c.args())
    torch.cuda.synchronize()
    assert int(c.status.item()) == 0 and (out[c.cu[-1]:] == 55.0).all()
    got = out.cpu().numpy()
    for s in (0, 1, 3, 6, 7, 8, len(q) - 1):
        for i in range(q[s]):
            want, _ = c.row(s, i, True)
            np.testing.assert_array_equal(got[c.cu[s] + i], want)
            if i % 16 == 0:
                Y, err = c.row(s, i, False)
                fine = np.isfinite(Y)
                assert (np.abs(got[c.cu[s] + i][fine] - Y[fine]) <= err[fine]).all()


@pytest.mark.parametrize("V", [500, 4097, 4098])
@pytest.mark.parametrize("tree", [False, True])
def test_counts_under_clear_bits_are_not_read(ts, V, tree):
    """A state whose bits were cleared and whose counts were left: drafted tokens, and
    neighbours of tokens that were met."""
    c = Case([6, 20], V, BF, seed=V, tree=tree, n_bias=4, masks="shared")
    c.counts = np.where(c.seen, c.counts, c.rng.integers(1, 50, c.counts.shape)).astype(np.int32)
    if tree:
        c.seen[:, c.tokens[1::2]] = False
        c.seen[:, 5] = False
    assert (c.counts[~c.seen] > 0).any()
    c.run(ts)


@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("counts", [False, True])
@pytest.mark.parametrize("n_bias", [0, 1, 700])
@pytest.mark.parametrize("masks", ["none", "shared", "each"])
def test_parts(ts, tree, counts, n_bias, masks):
    Case([5, 1, 12], 6000, BF, seed=n_bias, tree=tree, counts=counts, n_bias=n_bias,
         masks=masks).run(ts, masked_value=-1e30 if n_bias else -np.inf)


def test_nothing_asked_is_a_copy_in_fp32(ts):
    for dtype in (F32, BF, FP):
        for V in (777, 8192):
            c = Case([3, 4], V, dtype, seed=1)
            out = ts.ts_logits_process(c.logits, i32(c.cu))
            assert torch.equal(out, c.logits.float())


@pytest.mark.parametrize("only", ["repetition", "frequency", "presence", "seen"])
def test_single_penalties(ts, only):
    c = Case([2, 6], 3001, FP, seed=2, tree=False)
    args = c.args()
    keep = {k: args[k] for k in ("seen", "counts")}
    if only != "seen":
        keep[only] = args[only]
    neutral = dict(rep=1.0, freq=0.0, pres=0.0)
    for k, name in (("rep", "repetition"), ("freq", "frequency"), ("pres", "presence")):
        if name != only:
            setattr(c, k, np.full(2, neutral[k], dtype=np.float32))
    c.check(ts.ts_logits_process(c.logits, i32(c.cu), **keep))


def test_paths_count_without_a_state(ts):
    c = Case([20, 64], 500, F32, seed=3)
    c.seen[:] = False
    args = c.args()
    args.pop("seen"), args.pop("counts")
    c.check(ts.ts_logits_process(c.logits, i32(c.cu), **args))


@pytest.mark.parametrize("V", [4096, 4099, 30000])
def test_in_place(ts, V):
    c = Case([9, 30], V, F32, seed=4, n_bias=5, masks="each", pad=4)
    want = ts.ts_logits_process(c.logits, i32(c.cu), **c.args())
    view = c.logits
    r = ts.ts_logits_process(view, i32(c.cu), out=view, **c.args())
    assert r is view and torch.equal(view, want)


def test_equal_ids_and_special_values(ts):
    """Of equal ids the last bias counts; infinities and NaN follow the arithmetic,
    and a masked place hides them."""
    c = Case([2], 4500, F32, seed=5, tree=False, counts=True)
    c.bias_ids = np.array([[7, 7, 4499, 7, -1, 4499, 100]], dtype=np.int32)
    c.bias = np.array([[1, 2, 3, -5, 9, np.inf, -np.inf]], dtype=np.float32)
    c.run(ts)
    x = c.logits
    c.seen[0, :8], c.counts[0, :8] = True, 2
    x[0, :4] = torch.tensor([float("nan"), float("inf"), float("-inf"), 0.0])
    x[1, :4] = torch.tensor([-0.0, 3e38, -3e38, 1e-40])
    c.rep[:], c.freq[:], c.pres[:] = 1.25, 0.5, 0.25
    out = ts.ts_logits_process(x, i32(c.cu), **c.args())
    got = out.cpu().numpy()
    for i in range(2):
        with np.errstate(all="ignore"):
            want, _ = c.row(0, i, True)
        np.testing.assert_array_equal(got[i], want)
    words = cuda(lo.pack(np.zeros((1, 4500), dtype=bool)))
    hidden = ts.ts_logits_process(x, i32(c.cu), mask=words, mask_rows=i32([0, -1]), masked_value=-7.0)
    assert (hidden[0] == -7.0).all() and torch.equal(hidden[1], x[1])
    # no grammar at all: a table without masks
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    free = ts.ts_logits_process(x, i32(c.cu), mask=words[:0], mask_rows=i32([-1, -1]), status=status)
    assert torch.equal(free[1], x[1]) and int(status.item()) == 0
    ts.ts_logits_process(x, i32(c.cu), mask=words[:0], mask_rows=i32([-1, 0]), status=status)
    assert int(status.item()) == 1


def test_large_vocabulary_and_many_rows(ts):
    c = Case([1] * 70, 262144, BF, seed=6, tree=False, n_bias=300, masks="shared")
    c.run(ts)
    c = Case([0] * 5 + [1] * 900, 100, FP, seed=7, tree=True, n_bias=3)
    c.run(ts)


@pytest.mark.parametrize("what", ["cu", "long tree", "parent", "token", "bias", "mask row", "repetition"])
def test_bad_device_data_is_reported(ts, what):
    """A status and no access outside; the other sequence's rows are as they should be."""
    for V in (5000, 8192):
        c = Case([6, 70 if what == "long tree" else 8], V, BF, seed=8, n_bias=4, masks="shared",
                 extra=4, tree=what != "long tree")
        args, cu = c.args(), i32(c.cu)
        if what == "cu":
            for bad in ([0, 6, 10 ** 6], [0, -5, 14], [0, 6, 3]):
                c.status.zero_()
                ts.ts_logits_process(c.logits, i32(bad), status=c.status, **args)
                assert int(c.status.item()) == 1
            continue
        if what == "long tree":
            args.update(tree_tokens=cuda(c.tokens), parents=i32([-1] + [0] * 5 + [-1] + [0] * 69 + [0] * 4))
        if what == "parent":
            args["parents"][9] = 7
        if what == "token":
            args["tree_tokens"][9] = V
        if what == "bias":
            args["bias_ids"][1, 2] = V
        if what == "mask row":
            args["mask_rows"][9] = 3
        if what == "repetition":
            args["repetition"][1] = 0.0
        out = ts.ts_logits_process(c.logits, cu, status=c.status, **args)
        torch.cuda.synchronize()
        assert int(c.status.item()) == 1
        if what == "long tree":
            continue
        for i in range(6):
            want, _ = c.row(0, i, True)
            np.testing.assert_array_equal(out[i].cpu().numpy(), want)


def test_the_sequence_beside_a_long_tree(ts):
    for V in (5000, 8192):
        c = Case([6, 70], V, BF, seed=8, n_bias=4, masks="shared")
        par = [-1] + [0] * 5 + [-1] + [0] * 69
        out = ts.ts_logits_process(c.logits, i32(c.cu), status=c.status,
                                   **{**c.args(), "parents": i32(par)})
        torch.cuda.synchronize()
        assert int(c.status.item()) == 1
        c.parents = i32(par)
        got = out.cpu().numpy()
        for i in range(6):
            want, _ = c.row(0, i, True)
            np.testing.assert_array_equal(got[i], want)


@pytest.mark.parametrize("V", [5000, 5001])
@pytest.mark.parametrize("bad,good", [([0, 6, 10 ** 6], 1), ([0, 6, 3], 1), ([0, 6, -1], 1),
                                      ([0, 6, 14, 2], 2), ([2, 8, 14, 5, 5, 5], 2)])
def test_sequences_in_front_of_bad_offsets(ts, V, bad, good):
    """Sequences in front of an offset out of its range or order keep their rows,
    masks and penalties."""
    ns = len(bad) - 1
    c = Case([3] * ns, V, BF, seed=8, n_bias=4, masks="shared", extra=20 - 3 * ns)
    check_in_front(ts, c, bad, range(good))


@pytest.mark.parametrize("tail", [[2], [9, 6, 6], [-7]])
def test_blocks_of_rows_in_front_of_bad_offsets(ts, tail):
    """Blocks of several rows, which begin in front of the last offset or behind it."""
    c = Case([30] * 14 + [64] * 14 + [5] * len(tail), 4098, F32, seed=9, n_bias=4, masks="shared")
    assert c.n * 3 // (152 * 6) > 1
    check_in_front(ts, c, c.cu[:29] + tail, (0, 1, 13, 14, 15, 26, 27), same=True)


def check_in_front(ts, c, bad, seqs, same=False):
    """The rows of `seqs`; same: those are where the case has them, trees and all."""
    c.cu = bad
    if not same:
        par = [0] * c.n
        for s in seqs:
            par[bad[s]:bad[s + 1]] = range(-1, bad[s + 1] - bad[s] - 1)
        c.parents = i32(par)
    out = torch.full((c.n, c.V), 55.0, device="cuda")
    ts.ts_logits_process(c.logits, i32(bad), out=out, status=c.status, **c.args())
    torch.cuda.synchronize()
    assert int(c.status.item()) == 1
    assert (out[:bad[0]] == 55.0).all()
    got = out.cpu().numpy()
    for s in seqs:
        for i in range(bad[s + 1] - bad[s]):
            want, _ = c.row(s, i, True)
            np.testing.assert_array_equal(got[bad[s] + i], want)


@pytest.mark.parametrize("V", [3000, 8192])
@pytest.mark.parametrize("n_seq,lead", [(3, 1), (3, 2), (400, 1), (400, 399)])
def test_sequences_of_a_larger_batch(ts, V, n_seq, lead):
    """The last of a batch's sequences alone: rows in front of the first and behind the
    last are left as they were, whatever their masks, tokens and parents say."""
    c = Case([5 if s == 1 else 3 for s in range(n_seq)], V, F32, seed=lead, extra=6, n_bias=3,
             masks="shared")
    args = c.args()
    for name in ("seen", "counts", "repetition", "frequency", "presence", "bias_ids", "bias"):
        args[name] = args[name][lead:].contiguous()
    for name, what in (("mask_rows", 99), ("tree_tokens", -3), ("parents", 77)):
        args[name] = args[name].clone()
        args[name][:c.cu[lead]] = what
        args[name][c.cu[-1]:] = what
    out = torch.full((c.n, V), 55.0, device="cuda")
    ts.ts_logits_process(c.logits, i32(c.cu[lead:]), out=out, status=c.status, **args)
    torch.cuda.synchronize()
    assert int(c.status.item()) == 0
    assert (out[:c.cu[lead]] == 55.0).all() and (out[c.cu[-1]:] == 55.0).all()
    got = out.cpu().numpy()
    for s in sorted({lead, (lead + n_seq) // 2, n_seq - 1}):
        for i in range(c.q_lens[s]):
            want, _ = c.row(s, i, True)
            np.testing.assert_array_equal(got[c.cu[s] + i], want)


def test_logits_replay_and_streams(ts):
    c = Case([8, 8], 9000, BF, seed=9, n_bias=6, masks="each")
    args, cu = c.args(), i32(c.cu)
    out = torch.empty(c.n, c.V, device="cuda")
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    own = ts.ts_logits_process(c.logits, cu, stream=st, **args)
    st.synchronize()
    c.check(own)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ts.ts_logits_process(c.logits, cu, out=out, status=c.status, **args)
    for i in range(2):
        c.tokens = c.rng.integers(0, c.V, c.n).astype(np.int32)
        c.seen = c.rng.random((2, c.V)) < 0.2
        c.counts = (c.rng.integers(0, 9, (2, c.V)) * c.seen).astype(np.int32)
        c.q_lens, c.cu = ([3, 13], [0, 3, 16]) if i else ([8, 8], [0, 8, 16])
        c.parents.copy_(parents_of(c.q_lens, "mixed", seed=i))
        cu.copy_(i32(c.cu))
        args["tree_tokens"].copy_(cuda(c.tokens))
        args["seen"].copy_(cuda(lo.pack(c.seen)))
        args["counts"].copy_(cuda(c.counts))
        g.replay()
        torch.cuda.synchronize()
        assert int(c.status.item()) == 0
        c.check(out)


def test_calls_on_two_streams_at_once(ts):
    """Two batches' logits and counts on two streams, back and forth, without waits."""
    cases = [Case([5, 20], 50000, dtype, seed=20 + i, n_bias=30, masks="each")
             for i, dtype in enumerate((BF, F32))]
    args = [(c.logits, i32(c.cu), c.args()) for c in cases]
    tokens = [cuda(c.rng.integers(0, c.V, (2, 4000)).astype(np.int32)) for c in cases]
    lens = i32([4000, 17])
    states = [(torch.zeros((2, (c.V + 31) // 32), dtype=torch.int32, device="cuda"),
               torch.zeros((2, c.V), dtype=torch.int32, device="cuda")) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    outs = [[], []]
    for i in range(6):
        for k, st in enumerate(streams):
            outs[k].append(ts.ts_logits_process(args[k][0], args[k][1], stream=st, **args[k][2]))
            ts.ts_token_counts(tokens[k], lens, cases[k].V, *states[k], reset=i % 3 == 0, stream=st)
    torch.cuda.synchronize()
    for k, c in enumerate(cases):
        c.check(outs[k][0])
        assert all(torch.equal(outs[k][0], x) for x in outs[k][1:])
        C = np.stack([np.bincount(t[:m], minlength=c.V) for t, m in
                      zip(tokens[k].cpu().numpy(), (4000, 17))])
        np.testing.assert_array_equal(states[k][1].cpu().numpy(), 3 * C)


def test_an_empty_batch_of_rows(ts):
    out = ts.ts_logits_process(torch.empty(0, 100, device="cuda"), i32([0]))
    assert out.shape == (0, 100)


def test_logits_refusals_of_the_binding(ts):
    x, cu = torch.zeros(4, 100, device="cuda"), i32([0, 4])
    with pytest.raises(ValueError):
        ts.ts_logits_process(x.t(), i32([0, 100]))                  # values not dense
    with pytest.raises(ValueError):
        ts.ts_logits_process(x[0:1].expand(4, 100), cu)             # rows on top of one another
    with pytest.raises(TypeError):
        ts.ts_logits_process(x.double(), cu)
    with pytest.raises(ValueError):
        ts.ts_logits_process(x, cu, bias_ids=i32([[1]]))
    with pytest.raises(ValueError):
        ts.ts_logits_process(x, cu, seen=i32([[1]]))                # too few words
    with pytest.raises(TypeError):
        ts.ts_logits_process(x, cu, repetition=i32([1]))
    with pytest.raises(ValueError):
        ts.ts_logits_process(x, cu, out=torch.zeros(4, 101, device="cuda"))
    with pytest.raises(ts.TsError):
        ts.ts_logits_process(x, cu, counts=torch.zeros(1, 100, dtype=torch.int32, device="cuda"))
    big = torch.zeros(8, 100, device="cuda")
    with pytest.raises(ts.TsError):
        ts.ts_logits_process(big[:4], cu, out=big[2:6])


# ------------------------------------------------------------------ counts
@pytest.mark.parametrize("V", [1, 32, 45, 1000, 8192, 70001, 262144])
@pytest.mark.parametrize("m", [0, 1, 3, 300, 5000])
@pytest.mark.parametrize("reset", [False, True])
def test_counts(ts, V, m, reset):
    rng = np.random.default_rng(V + m)
    lens = [m, 0, (m + 1) // 2, m]
    tokens = (rng.random((4, m)) ** 4 * V).astype(np.int32)
    if m > 2:
        tokens[3] = V - 1                                # one token many times
    c0 = rng.integers(0, 5, (4, V)).astype(np.int32)
    s0 = rng.random((4, V)) < 0.2
    for prompt in (False, True):
        for with_counts in (True, False):
            status = torch.zeros(1, dtype=torch.int32, device="cuda")
            counts, seen = cuda(c0), cuda(lo.pack(s0))
            ts.ts_token_counts(cuda(tokens), i32(lens), V, seen, counts if with_counts else None,
                               reset=reset, prompt=prompt, status=status)
            C, S = lo.count_tokens(tokens, lens, V, c0, s0, reset, prompt)
            assert int(status.item()) == 0
            np.testing.assert_array_equal(lo.unpack(seen.cpu().numpy(), V), S)
            np.testing.assert_array_equal(seen.cpu().numpy(), lo.pack(S))
            np.testing.assert_array_equal(counts.cpu().numpy(), C if with_counts else c0)


@pytest.mark.parametrize("reset", [False, True])
def test_counts_of_many_sequences_and_a_long_one(ts, reset):
    rng = np.random.default_rng(3)
    for n, m, V in ((900, 3, 40), (2, 100_000, 130_000)):
        tokens = (rng.random((n, m)) ** 3 * V).astype(np.int32)
        lens = rng.integers(0, m + 1, n).tolist()
        counts = torch.full((n, V), 2, dtype=torch.int32, device="cuda")
        seen = torch.zeros((n, (V + 31) // 32), dtype=torch.int32, device="cuda")
        ts.ts_token_counts(cuda(tokens), i32(lens), V, seen, counts, reset=reset)
        C = np.stack([np.bincount(t[:k], minlength=V) for t, k in zip(tokens, lens)])
        np.testing.assert_array_equal(counts.cpu().numpy(), C + (0 if reset else 2))
        np.testing.assert_array_equal(lo.unpack(seen.cpu().numpy(), V), C > 0)


@pytest.mark.parametrize("reset", [False, True])
def test_counts_report_bad_tokens_and_lengths(ts, reset):
    for V in (50, 40000):
        tokens = np.array([[1, 2, -1, 3], [4, V, 5, 6], [7, 8, 9, 10]], dtype=np.int32)
        for lens, good in (([4, 4, 4], [[1, 2, 3], [4, 5, 6], [7, 8, 9, 10]]),
                           ([2, 1, 5], [[1, 2], [4], [7, 8, 9, 10]]),
                           ([2, -1, 4], [[1, 2], [], [7, 8, 9, 10]])):
            counts = torch.zeros((3, V), dtype=torch.int32, device="cuda")
            seen = torch.zeros((3, (V + 31) // 32), dtype=torch.int32, device="cuda")
            status = torch.zeros(1, dtype=torch.int32, device="cuda")
            ts.ts_token_counts(cuda(tokens), i32(lens), V, seen, counts, reset=reset, status=status)
            assert int(status.item()) == 1
            for s in range(3):
                assert torch.nonzero(counts[s]).flatten().tolist() == good[s]


def test_counts_replay_and_refusals(ts):
    tokens, lens = torch.zeros((2, 6), dtype=torch.int32, device="cuda"), i32([0, 0])
    counts = torch.zeros((2, 300), dtype=torch.int32, device="cuda")
    seen = torch.zeros((2, 10), dtype=torch.int32, device="cuda")
    ts.ts_token_counts(tokens, lens, 300, seen, counts)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ts.ts_token_counts(tokens, lens, 300, seen, counts)
    C, S = np.zeros((2, 300), int), np.zeros((2, 300), bool)
    rng = np.random.default_rng(4)
    for _ in range(3):
        t, m = rng.integers(0, 300, (2, 6)), rng.integers(0, 7, 2).tolist()
        tokens.copy_(cuda(t, torch.int32))
        lens.copy_(i32(m))
        g.replay()
        C, S = lo.count_tokens(t, m, 300, C, S, False, False)
    np.testing.assert_array_equal(counts.cpu().numpy(), C)
    np.testing.assert_array_equal(lo.unpack(seen.cpu().numpy(), 300), S)
    with pytest.raises(ValueError):
        ts.ts_token_counts(tokens, lens, 300, seen[:, :9].contiguous(), counts)
    with pytest.raises(ValueError):
        ts.ts_token_counts(tokens[:, ::2], lens, 300, seen, counts)
    with pytest.raises(TypeError):
        ts.ts_token_counts(tokens.long(), lens, 300, seen, counts)


# ------------------------------------------------------------------ a step of all calls
@pytest.mark.parametrize("dtype", [BF, FP], ids=["bf16", "fp16"])
def test_steps_of_several_streams(ts, dtype):
    """Three steps of two streams: trees written into the pages, verified, their
    logits processed, sampled and accepted, the accepted rows moved and counted,
    with lengths that stay on the device.  The cache, the state and the next
    step's attention are those of a stream that had only ever held the accepted
    tokens."""
    ns, T, V, Hq, Hkv, d, ps, n_layers = 2, 13, 1500, 8, 2, 64, 16, 2
    rng = np.random.default_rng(11)
    g = torch.Generator(device="cuda").manual_seed(3)
    n_pages, width = 40, 12
    shape = (n_layers, n_pages, Hkv, ps, d)
    k, v = (torch.zeros(shape, dtype=dtype, device="cuda") for _ in range(2))
    bounds = [torch.zeros((n_layers, n_pages, Hkv, d), dtype=dtype, device="cuda") for _ in range(2)]
    table = i32(rng.permutation(n_pages)[:ns * width].reshape(ns, width).tolist())
    freqs, _ = ts.ts_rope_frequencies(d)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    emb_k, emb_v, emb_q = (torch.randn(V, n_layers, h, d, generator=g, device="cuda").to(dtype)
                           for h in (Hkv, Hkv, Hq))
    head = torch.randn(Hq * d, V, generator=g, device="cuda") * 0.2
    prompts = [rng.integers(0, V, 37).tolist(), rng.integers(0, V, 21).tolist()]
    pad = np.zeros((ns, 37), dtype=np.int32)
    for s in range(ns):
        pad[s, :len(prompts[s])] = prompts[s]
    counts = torch.ones((ns, V), dtype=torch.int32, device="cuda")
    seen = torch.ones((ns, (V + 31) // 32), dtype=torch.int32, device="cuda")
    ts.ts_token_counts(cuda(pad), i32([37, 21]), V, seen, counts, reset=True, prompt=True,
                       status=status)
    cu = i32([0, 37, 58])
    toks = torch.tensor(prompts[0] + prompts[1], device="cuda")
    lens = i32([37, 21])

    def write(toks, cu, lens, positions):
        out = []
        for l in range(n_layers):
            out.append(ts.ts_paged_rope_append(
                emb_q[toks, l].contiguous(), emb_k[toks, l].contiguous(), emb_v[toks, l].contiguous(),
                cu, lens, table, k[l], v[l], freqs, positions=positions, key_min=bounds[0][l],
                key_max=bounds[1][l], status=status))
        return out

    write(toks, cu, lens, None)
    layers, blayers = ts.commit_pointer_table(k, v), ts.commit_pointer_table(*bounds)
    cu = i32([0, T, 2 * T])
    rep, freq = torch.full((ns,), 1.2, device="cuda"), torch.full((ns,), 0.1, device="cuda")
    roots = [int(p[-1]) for p in prompts]
    # the root's row is written again as the tree's first node
    lens = lens - 1
    history = [list(p) for p in prompts]
    generated = [[] for _ in range(ns)]
    likely = i32([[0, 1, 2, 3]] * ns)
    push = torch.full((ns, 4), 30.0, device="cuda")
    longest = 0
    for step in range(3):
        par = parents_of([T] * ns, "ternary")
        depth = np.array([len(p) - 1 for p in po.root_paths(par[:T].tolist())])
        # biases make the first four tokens likely, and drafts of them get accepted
        tree = np.array([[(i + s + step) % 4 for i in range(T)] for s in range(ns)], dtype=np.int32)
        tree[:, 0] = roots
        tree_t = cuda(tree)
        positions = (lens[:, None] + cuda(depth, torch.int32)[None]).reshape(-1).contiguous()
        toks = tree_t.reshape(-1).long()
        new_lens = lens + T
        q = write(toks, cu, new_lens, positions)
        for l in range(n_layers):
            o, lse = ts.ts_paged_tree_attention(q[l], k[l], v[l], cu, new_lens, table, par, T,
                                                status=status)
            # what a stream that holds the accepted tokens alone would attend to
            L = lens.tolist()
            O = po.tree_attention(pu.f64(q[l]), pu.f64(k[l]), pu.f64(v[l]), [0, T, 2 * T],
                                  [x + T for x in L], table.cpu().numpy(), par.cpu().numpy())
            pu.check_attention(o, lse, O, dtype, d, p_round=2.0 ** -8)
        logits = o.float().reshape(ns * T, -1) @ head
        allowed = rng.random((ns * T, V)) < 0.5
        allowed[:, :4] = True
        y = ts.ts_logits_process(logits, cu, seen=seen, counts=counts, repetition=rep, frequency=freq,
                                 tree_tokens=toks.int(), parents=par, bias_ids=likely, bias=push,
                                 mask=cuda(lo.pack(allowed)),
                                 status=status)
        u = torch.rand(ns * T, generator=g, device="cuda")
        sampled, path, n_path = [], [], []
        for s in range(ns):
            a = s * T
            assert history[s][-1] == int(tree[s, 0])
            r = ts.ts_penalized_sample_accept(y[a:a + T], tree_t[s].contiguous(), par[a:a + T],
                                              i32(history[s]), 0, 1.0, 1.0, 0.9, 0.05, u[a:a + T],
                                              status=status)
            sampled.append(r[0]), path.append(r[1]), n_path.append(r[2])
            got = r[0].long()
            assert allowed[np.arange(a, a + T), got.cpu().numpy()].all()
        path, n_path = torch.stack(path), torch.cat(n_path)
        lens2 = ts.ts_paged_kv_commit(k, v, cu, new_lens, table, path, n_path, key_min=bounds[0],
                                      key_max=bounds[1], table=layers, bounds_table=blayers,
                                      status=status)
        # (what stands behind a path is not written)
        took = torch.gather(torch.stack(sampled), 1, path.clamp(0, T - 1).long())
        ts.ts_token_counts(took.contiguous(), n_path, V, seen, counts, status=status)
        torch.cuda.synchronize()
        assert int(status.item()) == 0
        for s in range(ns):
            m = int(n_path[s])
            longest = max(longest, m)
            new = took[s, :m].tolist()
            assert new[:-1] == tree[s][path[s, 1:m].cpu().numpy()].tolist()
            history[s] += new
            generated[s] += new
            roots[s] = new[-1]
            assert int(lens2[s]) == len(history[s]) - 1
            C = np.bincount(generated[s], minlength=V)
            np.testing.assert_array_equal(counts[s].cpu().numpy(), C)
            S = np.zeros(V, dtype=bool)
            S[history[s]] = True
            np.testing.assert_array_equal(lo.unpack(seen[s].cpu().numpy(), V), S)
            # the cache holds the history's rows: rotated again from the tokens
            rows = torch.tensor(history[s][:-1], device="cuda")
            m = len(rows)
            fresh = [torch.zeros((1, width, Hkv, ps, d), dtype=dtype, device="cuda") for _ in range(2)]
            own = torch.arange(width, dtype=torch.int32, device="cuda")[None].contiguous()
            for l in range(n_layers):
                ts.ts_paged_rope_append(emb_q[rows, l].contiguous(), emb_k[rows, l].contiguous(),
                                        emb_v[rows, l].contiguous(), i32([0, m]), i32([m]), own,
                                        fresh[0][0], fresh[1][0], freqs)
                for x, f in ((k[l], fresh[0][0]), (v[l], fresh[1][0])):
                    a = x[table[s].long()].permute(0, 2, 1, 3).reshape(-1, Hkv, d)[:m]
                    b = f.permute(0, 2, 1, 3).reshape(-1, Hkv, d)[:m]
                    assert torch.equal(a, b)
                # the bounds hold every row of a page
                full = (m + ps - 1) // ps
                for pg in range(full):
                    ph = int(table[s, pg])
                    held = k[l, ph, :, :min(ps, m - pg * ps)].float()
                    assert (bounds[0][l, ph].float() <= held.amin(1)).all()
                    assert (bounds[1][l, ph].float() >= held.amax(1)).all()
        lens = lens2
    assert longest > 1                     # some draft was accepted
