"""Draft trees over the paged cache and node logits, host side: the oracle's pins
and the calls' refusals (no call here reaches a GPU)."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import logits_oracle as lo
from oracle import paged_oracle as po
from oracle import ts_oracle as orc


@pytest.fixture(scope="module")
def ts():
    import self_speculative_ultra_gb300 as ts
    ts.build()
    return ts


P = ctypes.c_void_p(256)
FAR = ctypes.c_void_p(1 << 40)
ODD = ctypes.c_void_p(8)


# ------------------------------------------------------------------ oracle pins
def _pool(rng, Hkv=2, d=8, ps=16, n_pages=7):
    return rng.standard_normal((n_pages, Hkv, ps, d)), rng.standard_normal((n_pages, Hkv, ps, d))


def test_a_chain_is_causal_and_a_tree_is_the_contiguous_one():
    rng = np.random.default_rng(0)
    k, v = _pool(rng)
    table = np.array([[4, 1, 6], [2, 0, 5]])
    cu, lens = [0, 9, 20], [37, 11]
    q = rng.standard_normal((20, 4, 8))
    chain = [i - 1 for i in range(9)] + [i - 1 for i in range(11)]
    for a, b in zip(po.tree_attention(q, k, v, cu, lens, table, chain),
                    po.attention(q, k, v, cu, lens, table)):
        np.testing.assert_allclose(a, b, rtol=1e-12, atol=1e-12)
    par = [-1, 0, 0, 1, 1, 2, 5, 0, 7]
    O, LSE, *_ = po.tree_attention(q[:9], k, v, [0, 9], lens[:1], table[:1], par)
    kc = np.stack([po.sequence_rows(k, table[0], 37, h) for h in range(2)])
    vc = np.stack([po.sequence_rows(v, table[0], 37, h) for h in range(2)])
    o, lse, _ = orc.verify_attention(q[:9], kc, vc, 28, np.array(par), 1)
    np.testing.assert_allclose(O, o, rtol=1e-12, atol=1e-12)
    np.testing.assert_allclose(LSE, lse, rtol=1e-12, atol=1e-12)


def test_commit_oracle():
    rng = np.random.default_rng(1)
    k, v = _pool(rng)
    mn, mx = k.min(2) - 1, k.max(2) + 1
    table = np.array([[4, 1, 6]])
    # rows 13 .. 21 are the tree: pages 4 (13..15) and 1 (16..21)
    k2, v2, mn2, mx2, new = po.kv_commit(k, v, mn, mx, [0, 9], [22], table, [[0, 2, 5, 8]], [4])
    assert new == [17]
    for t, a in enumerate([0, 2, 5, 8]):
        src, dst = 13 + a, 13 + t
        np.testing.assert_array_equal(k2[table[0][dst // 16], :, dst % 16],
                                      k[table[0][src // 16], :, src % 16])
    np.testing.assert_array_equal(mn2[1], k2[1, :, 0])        # row 16 alone: the page started over
    np.testing.assert_array_equal(mx2[1], k2[1, :, 0])
    np.testing.assert_array_equal(mn2[4], np.minimum(mn[4], k2[4, :, 13:].min(1)))   # widened
    changed = np.argwhere((k2 != k).any((1, 3)))
    assert changed.tolist() == [[1, 0], [4, 14], [4, 15]]


def test_logits_oracle_by_hand():
    x = np.array([2.0, -2.0, 1.0, 4.0, 0.5, -1.0], dtype=np.float32)
    seen = np.array([1, 1, 0, 0, 0, 0], dtype=bool)
    counts = np.array([3, 0, 9, 0, 0, 0])
    allowed = np.array([1, 1, 1, 1, 1, 0], dtype=bool)
    for literal in (False, True):
        y, err = lo.process_row(x, {2: 1.5, 4: -0.25}, seen, counts, [3, 3], 2.0, 0.5, 0.25, allowed,
                                -np.inf, literal)
        # seen three times; seen in the prompt alone; biased; drafted twice; biased; not allowed
        np.testing.assert_array_equal(y, [1.0 - 1.5 - 0.25, -4.0, 2.5, 2.0 - 1.0 - 0.25, 0.25, -np.inf])
        assert err[5] == 0 and (err[:5] >= 0).all() and err[0] < 1e-6


def test_packing_round_trip_and_counts():
    rng = np.random.default_rng(2)
    bits = rng.random((3, 77)) < 0.5
    bits[:, 31] = True                                        # the word's sign bit
    assert lo.pack(bits).dtype == np.int32
    np.testing.assert_array_equal(lo.unpack(lo.pack(bits), 77), bits)
    c, s = lo.count_tokens([[1, 1, 3], [0, 2, 2]], [3, 1], 4, np.ones((2, 4), int),
                           np.zeros((2, 4), bool), False, False)
    assert c.tolist() == [[1, 3, 1, 2], [2, 1, 1, 1]]
    assert s.tolist() == [[False, True, False, True], [True, False, False, False]]
    c, s = lo.count_tokens([[1]], [1], 4, np.ones((1, 4), int), np.ones((1, 4), bool), True, True)
    assert c.sum() == 0 and s.tolist() == [[False, True, False, False]]


# ------------------------------------------------------------------ refusals
def _tree(ts, **kw):
    a = dict(q=P, k=P, v=P, n=100, Hq=32, Hkv=8, d=128, cu=P, lens=P, n_seq=2, table=P, maxp=4,
             ps=64, n_pages=8, par=P, max_q=64, max_kv=0, o=P, lse=P, ws=None, nb=0, flags=0,
             status=None, stream=None)
    a.update(kw)
    return ts.lib().ts_paged_tree_attention(*a.values())


def test_tree_attention_refusals(ts):
    assert _tree(ts, n=0, q=None, k=None, v=None, o=None, par=None) == 0     # nothing to do
    assert _tree(ts, n_seq=0, cu=None, lens=None, table=None, par=None) == 0
    for kw in (dict(par=None), dict(q=None), dict(k=None), dict(v=None), dict(o=None), dict(cu=None),
               dict(lens=None), dict(table=None), dict(max_q=0), dict(n=63), dict(n=-1),
               dict(Hq=30), dict(maxp=0), dict(n_pages=0), dict(flags=2), dict(q=ODD), dict(o=ODD)):
        assert _tree(ts, **kw) == 1, kw
    for kw in (dict(max_q=65), dict(d=96), dict(ps=48), dict(Hq=2048), dict(maxp=1 << 20),
               dict(n_pages=1 << 30), dict(n_seq=(1 << 20) + 1)):
        assert _tree(ts, **kw) == 2, kw
    need = ts.lib().ts_paged_tree_attention_workspace_bytes(100, 2, 32, 8, 128, 1600, 64, 64, 0)
    assert need > 0
    big = dict(maxp=1600, n_pages=4000)
    assert _tree(ts, **big) == 5
    assert _tree(ts, ws=P, nb=need - 1, **big) == 5
    assert _tree(ts, ws=ODD, nb=need, **big) == 5
    f = ts.lib().ts_paged_tree_attention_workspace_bytes
    assert f(100, 2, 32, 8, 128, 1600, 64, 65, 0) == 0
    assert f(0, 2, 32, 8, 128, 1600, 64, 64, 0) == 0


def _commit(ts, **kw):
    a = dict(n_layers=2, k=P, v=P, Hkv=8, d=128, cu=P, lens=P, n_seq=2, table=P, maxp=4, ps=64,
             n_pages=8, path=P, stride=5, n_path=P, mn=None, mx=None, new=FAR, flags=0, status=None,
             stream=None)
    a.update(kw)
    return ts.lib().ts_paged_kv_commit(*a.values())


def test_commit_refusals(ts):
    assert _commit(ts, n_layers=0, k=None, v=None) == 0
    assert _commit(ts, n_seq=0, cu=None, lens=None, table=None, path=None) == 0
    for kw in (dict(k=None), dict(v=None), dict(path=None), dict(n_path=None), dict(cu=None),
               dict(lens=None), dict(table=None), dict(n_layers=-1), dict(Hkv=0), dict(stride=0),
               dict(mn=P), dict(mx=P), dict(flags=2), dict(maxp=0), dict(n_pages=0), dict(n_seq=-1)):
        assert _commit(ts, **kw) == 1, kw
    # the lengths in place, or one of them
    assert _commit(ts, new=P) == 1 and _commit(ts, new=ctypes.c_void_p(260)) == 1
    assert "overlap" in ts.ts_last_error()
    for kw in (dict(stride=65), dict(d=96), dict(ps=256), dict(n_pages=1 << 30),
               dict(n_layers=1 << 28), dict(Hkv=1 << 20, n_pages=1 << 10)):
        assert _commit(ts, **kw) == 2, kw


def _counts(ts, **kw):
    a = dict(tokens=P, stride=8, lens=P, n_seq=2, V=1000, counts=P, seen=P, flags=0, status=None,
             stream=None)
    a.update(kw)
    return ts.lib().ts_token_counts(*a.values())


def test_counts_refusals(ts):
    assert _counts(ts, n_seq=0, tokens=None, lens=None, seen=None) == 0
    assert _counts(ts, stride=0, tokens=None) == 0
    for kw in (dict(tokens=None), dict(lens=None), dict(seen=None), dict(V=0), dict(n_seq=-1),
               dict(stride=-1), dict(flags=4)):
        assert _counts(ts, **kw) == 1, kw
    for kw in (dict(V=262145), dict(n_seq=(1 << 20) + 1), dict(stride=(1 << 25) + 1)):
        assert _counts(ts, **kw) == 2, kw


def _logits(ts, **kw):
    a = dict(x=P, row=1000, n=4, V=1000, cu=P, n_seq=2, tokens=P, par=P, counts=P, seen=P, rep=P,
             freq=P, pres=P, ids=P, bias=P, n_bias=3, mask=P, n_masks=4, rows=P,
             masked=float("-inf"), out=FAR, out_row=1000, flags=0, status=None, stream=None)
    a.update(kw)
    return ts.lib().ts_logits_process(*a.values())


def test_logits_refusals(ts):
    assert _logits(ts, n=0, x=None, out=None) == 0
    assert _logits(ts, n_seq=0, cu=None) == 0
    for kw in (dict(x=None), dict(out=None), dict(cu=None), dict(tokens=None), dict(par=None),
               dict(seen=None), dict(ids=None), dict(bias=None), dict(n_bias=-1), dict(n_masks=-1),
               dict(mask=None), dict(mask=None, rows=None), dict(rows=None, n_masks=3), dict(V=0), dict(n=-1), dict(n_seq=-1),
               dict(row=999), dict(out_row=999), dict(flags=3), dict(flags=4),
               dict(x=ctypes.c_void_p(257)), dict(out=ctypes.c_void_p((1 << 40) + 2)),
               dict(x=ctypes.c_void_p(257), flags=1)):
        assert _logits(ts, **kw) == 1, kw
    for kw in (dict(V=262145, row=262145, out_row=262145), dict(n=(1 << 20) + 1),
               dict(n_seq=(1 << 20) + 1), dict(n_bias=65536)):
        assert _logits(ts, **kw) == 2, kw
    # rows that would be overwritten before they are read
    same = ctypes.c_void_p(1 << 40)
    for kw in (dict(x=same, flags=1), dict(x=same, row=1008),
               dict(x=ctypes.c_void_p((1 << 40) + 4 * 3999)),
               dict(x=ctypes.c_void_p((1 << 40) - 4 * 3999))):
        assert _logits(ts, **kw) == 1, kw
        assert "overlap" in ts.ts_last_error()


def test_binding_refuses_what_is_not_on_a_gpu(ts):
    x = torch.zeros(4, 100)
    cu = torch.tensor([0, 4], dtype=torch.int32)
    with pytest.raises(TypeError):
        ts.ts_logits_process(x, cu)
    with pytest.raises(TypeError):
        ts.ts_token_counts(torch.zeros(1, 4, dtype=torch.int32), cu[:1], 100,
                           torch.zeros(1, 4, dtype=torch.int32))
    pool = torch.zeros(2, 3, 1, 16, 64, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        ts.ts_paged_kv_commit(pool, pool, cu, cu[:1], cu[None], cu[None], cu[:1])
    with pytest.raises(ValueError):
        ts.ts_paged_kv_commit([], [], cu, cu[:1], cu[None], cu[None], cu[:1])
    with pytest.raises(TypeError):
        ts.ts_paged_tree_attention(torch.zeros(4, 2, 64, dtype=torch.bfloat16), pool[0], pool[0], cu,
                                   cu[:1], cu[None], cu[:4], 4)
