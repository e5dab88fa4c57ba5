"""Paged-cache operators, host side: the oracle's pins, the rotary frequencies
and the calls' refusals (no call here reaches a GPU)."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import paged_oracle as po


@pytest.fixture(scope="module")
def ts():
    import self_speculative_ultra_gb300 as ts
    ts.build()
    return ts


SCALINGS = [dict(scaling="plain"), dict(scaling="linear", factor=4.0),
            dict(scaling="base", factor=8.0), dict(scaling="base", factor=1.0),
            dict(scaling="wavelength", factor=8.0, original_len=8192.0, low=1.0, high=4.0),
            dict(scaling="ramp", factor=16.0, original_len=4096.0, low=1.0, high=32.0)]


@pytest.mark.parametrize("kw", SCALINGS, ids=lambda k: k["scaling"])
@pytest.mark.parametrize("rot_dim,base", [(128, 10000.0), (64, 500000.0), (16, 10000.0), (2, 100.0)])
def test_rope_frequencies_match_their_formulas(ts, kw, rot_dim, base):
    if kw["scaling"] == "base" and rot_dim < 4:
        pytest.skip("a stretched base has no exponent at two columns")
    f, scale = ts.ts_rope_frequencies(rot_dim, base, device="cpu", **kw)
    F, S = po.rope_frequencies(rot_dim, base, **kw)
    assert f.dtype == torch.float64 and f.shape == (rot_dim // 2,)
    # a handful of 64-bit roundings: pow, one or two products, a blend
    np.testing.assert_allclose(f.numpy(), F, rtol=16 * np.finfo(np.float64).eps, atol=0)
    assert scale == pytest.approx(S, rel=2.0 ** -24)


def test_rope_frequencies_known_values(ts):
    f, scale = ts.ts_rope_frequencies(8, 16.0, device="cpu")
    np.testing.assert_allclose(f.numpy(), [1.0, 0.5, 0.25, 0.125], rtol=1e-15)
    assert scale == 1.0
    f, _ = ts.ts_rope_frequencies(8, 16.0, "linear", 4.0, device="cpu")
    np.testing.assert_allclose(f.numpy(), [0.25, 0.125, 0.0625, 0.03125], rtol=1e-15)
    # a pair of many turns keeps its frequency, one of few is divided
    f, _ = ts.ts_rope_frequencies(8, 16.0, "wavelength", 4.0, 2 * np.pi * 4, 1.0, 2.0, device="cpu")
    np.testing.assert_allclose(f.numpy(), [1.0, 0.5, 0.0625, 0.03125], rtol=1e-12)


def test_rope_frequencies_refusals(ts):
    out = (ctypes.c_double * 64)()
    f = ts.lib().ts_rope_frequencies
    ok = [128, 10000.0, 0, 1.0, 0.0, 1.0, 32.0, out, None]
    assert f(*ok) == 0
    for at, bad in [(0, 0), (0, 3), (0, 1026), (1, 1.0), (1, float("nan")), (2, 5), (2, -1),
                    (7, None)]:
        a = list(ok)
        a[at] = bad
        assert f(*a) == 1, (at, bad)
    for scaling, more in [(1, {3: 0.5}), (2, {3: 0.0}), (2, {0: 2, 3: 2.0}), (3, {4: 0.0}),
                          (3, {5: 0.0, 4: 10.0}), (4, {4: 10.0, 5: 4.0, 6: 4.0}),
                          (1, {3: float("inf")})]:
        a = list(ok)
        a[2] = scaling
        a[3] = 2.0
        for at, x in more.items():
            a[at] = x
        assert f(*a) == 1, (scaling, more)
    with pytest.raises(ValueError):
        ts.ts_rope_frequencies(128, scaling="other", device="cpu")


# ------------------------------------------------------------------ refusals
P = ctypes.c_void_p(256)
ODD = ctypes.c_void_p(8)


def _append(ts, **kw):
    a = dict(q=P, k=P, v=P, qs=32 * 128, ks=8 * 128, vs=8 * 128, n=4, Hq=32, Hkv=8, d=128, cu=P,
             lens=P, n_seq=2, table=P, maxp=4, ps=64, n_pages=8, pos=None, freqs=P, rot=128,
             scale=1.0, q_out=P, kp=P, vp=P, mn=None, mx=None, flags=0, status=None, stream=None)
    a.update(kw)
    return ts.lib().ts_paged_rope_append(*a.values())


def _attend(ts, **kw):
    a = dict(q=P, kp=P, vp=P, n=4, Hq=32, Hkv=8, d=128, cu=P, lens=P, n_seq=2, table=P, maxp=4,
             ps=64, n_pages=8, max_q=2, max_kv=0, o=P, lse=None, ws=P, nb=1 << 40, flags=0,
             status=None, stream=None)
    a.update(kw)
    return ts.lib().ts_paged_attention(*a.values())


def _select(ts, **kw):
    a = dict(q=P, mn=P, mx=P, n=4, Hq=32, Hkv=8, d=128, cu=P, lens=P, n_seq=2, table=P, maxp=4,
             ps=64, n_pages=8, top=2, sink=1, recent=1, pages=P, counts=P, ws=P, nb=1 << 40,
             flags=0, status=None, stream=None)
    a.update(kw)
    return ts.lib().ts_paged_select_pages(*a.values())


def _selected(ts, **kw):
    a = dict(q=P, kp=P, vp=P, n=4, Hq=32, Hkv=8, d=128, cu=P, lens=P, n_seq=2, table=P, maxp=4,
             ps=64, n_pages=8, pages=P, counts=P, n_sel=4, o=P, lse=None, ws=P, nb=1 << 40,
             flags=0, status=None, stream=None)
    a.update(kw)
    return ts.lib().ts_paged_attention_selected(*a.values())


@pytest.mark.parametrize("call", [_append, _attend, _select, _selected])
@pytest.mark.parametrize("kw,rc", [
    (dict(n=-1), 1), (dict(n_seq=-1), 1), (dict(Hq=0), 1), (dict(Hkv=0), 1), (dict(Hq=31), 1),
    (dict(Hq=2048), 2), (dict(d=96), 2), (dict(ps=48), 2), (dict(ps=8), 2), (dict(ps=256), 2),
    (dict(maxp=0), 1), (dict(n_pages=0), 1), (dict(maxp=(1 << 19) + 1), 2),
    (dict(n_seq=(1 << 20) + 1), 2), (dict(n_pages=1 << 24), 2),
    (dict(n=1 << 27), 2), (dict(cu=None), 1), (dict(lens=None), 1), (dict(table=None), 1),
    (dict(flags=64), 1), (dict(q=None), 1), (dict(q=ODD), 1)],
    ids=lambda x: str(x) if isinstance(x, int) else ",".join(x))
def test_shared_refusals(ts, call, kw, rc):
    assert call(ts, **kw) == rc
    assert ts.ts_last_error()


@pytest.mark.parametrize("call", [_append, _attend, _select, _selected])
def test_nothing_to_do_is_fine_without_tensors(ts, call):
    assert call(ts, n=0, q=None, cu=None, lens=None, table=None) == 0
    assert call(ts, n_seq=0, q=None, cu=None, lens=None, table=None) == 0


@pytest.mark.parametrize("kw,rc", [
    (dict(rot=-16), 1), (dict(rot=144), 1), (dict(rot=24), 2), (dict(freqs=None), 1),
    (dict(k=None), 1), (dict(vp=None), 1), (dict(mn=P), 1), (dict(mx=P), 1), (dict(qs=4095), 1),
    (dict(ks=1023), 1), (dict(vs=1028), 1), (dict(qs=4100), 1), (dict(kp=ODD), 1),
    (dict(mn=ODD, mx=P), 1), (dict(qs=8192), 1)], ids=lambda x: str(x) if isinstance(x, int) else ",".join(x))
def test_append_refusals(ts, kw, rc):
    # the last: q_out = q (the same address here) with a strided q
    if "qs" not in kw or kw["qs"] != 8192:
        kw = dict(kw, q_out=ctypes.c_void_p(512))
    assert _append(ts, **kw) == rc
    assert ts.ts_last_error()


@pytest.mark.parametrize("kw,rc", [
    (dict(max_q=0), 1), (dict(max_q=5), 1), (dict(kp=None), 1), (dict(o=None), 1),
    (dict(o=ODD), 1), (dict(flags=2), 1)], ids=str)
def test_attention_refusals(ts, kw, rc):
    assert _attend(ts, **kw) == rc
    assert ts.ts_last_error()


def test_workspace_refusals(ts):
    lib = ts.lib()
    need = lib.ts_paged_attention_workspace_bytes(4, 2, 32, 8, 128, 4000, 64, 2, 0)
    assert need > 0
    big = dict(maxp=4000, n_pages=4000)
    assert _attend(ts, ws=None, nb=0, **big) == 5
    assert _attend(ts, ws=ODD, **big) == 5
    assert _attend(ts, nb=need - 1, **big) == 5
    need = lib.ts_paged_select_workspace_bytes(4, 8, 4)
    assert need > 0
    assert _select(ts, nb=need - 1) == 5
    need = lib.ts_paged_selected_workspace_bytes(4, 32, 8, 128, 64, 4000)
    assert need > 0
    assert _selected(ts, n_sel=4000, nb=need - 1) == 5
    assert lib.ts_paged_attention_workspace_bytes(0, 2, 32, 8, 128, 4, 64, 2, 0) == 0
    assert lib.ts_paged_select_workspace_bytes(0, 8, 4) == 0
    assert lib.ts_paged_selected_workspace_bytes(4, 31, 8, 128, 64, 4) == 0


@pytest.mark.parametrize("kw,rc", [
    (dict(top=-1), 1), (dict(sink=-1), 1), (dict(recent=0), 1), (dict(top=1 << 25), 2),
    (dict(n=65536), 2), (dict(pages=None), 1), (dict(counts=None), 1), (dict(mx=ODD), 1)], ids=str)
def test_select_refusals(ts, kw, rc):
    assert _select(ts, **kw) == rc
    assert ts.ts_last_error()


@pytest.mark.parametrize("kw,rc", [
    (dict(n_sel=0), 1), (dict(n_sel=(1 << 19) + 1), 2), (dict(pages=None), 1), (dict(counts=None), 1)],
    ids=str)
def test_selected_refusals(ts, kw, rc):
    assert _selected(ts, **kw) == rc
    assert ts.ts_last_error()


def test_binding_refuses_host_tensors_and_wrong_types(ts):
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    kp = torch.zeros(3, 1, 16, 64, dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(TypeError):
        ts.ts_paged_attention(q, kp, kp, i, i[:1], i.view(1, 2), 1)
    with pytest.raises(TypeError):
        ts.ts_paged_rope_append(q, q[:, :1], q[:, :1], i, i[:1], i.view(1, 2), kp, kp,
                                torch.zeros(32, dtype=torch.float64))
    with pytest.raises(TypeError):
        ts.ts_paged_select_pages(q, kp[:, :, 0], kp[:, :, 0], i, i[:1], i.view(1, 2), 16, 1, 0, 1)


# ------------------------------------------------------------------ the oracle's pins
def test_oracle_rotation_turns_pairs():
    f = np.array([np.pi / 2, 0.0])
    x = np.array([1.0, 2.0, 3.0, 4.0, 5.0])
    # a quarter turn of the first pair, none of the second, the rest untouched
    np.testing.assert_allclose(po.rotate_row(x, 1, f, 1.0, False), [-3, 2, 1, 4, 5], atol=1e-15)
    np.testing.assert_allclose(po.rotate_row(x, 1, f, 1.0, True), [-2, 1, 3, 4, 5], atol=1e-15)
    np.testing.assert_allclose(po.rotate_row(x, 2, f, 2.0, True), [-2, -4, 6, 8, 5], atol=1e-14)


def test_oracle_rotation_keeps_relative_scores():
    rng = np.random.default_rng(0)
    f, _ = po.rope_frequencies(32)
    q, k = rng.normal(size=32), rng.normal(size=32)
    a = po.rotate_row(q, 900, f, 1.0, False) @ po.rotate_row(k, 850, f, 1.0, False)
    b = po.rotate_row(q, 60, f, 1.0, False) @ po.rotate_row(k, 10, f, 1.0, False)
    assert abs(a - b) < 1e-10


def test_oracle_attention_by_brute_force():
    rng = np.random.default_rng(1)
    kp, vp = rng.normal(size=(5, 1, 2, 4)), rng.normal(size=(5, 1, 2, 4))
    q = rng.normal(size=(3, 2, 4))
    table = np.array([[3, 0, 4]])
    o, lse, _, _ = po.attention(q, kp, vp, [0, 2], [5], table)
    k = np.stack([kp[3, 0, 0], kp[3, 0, 1], kp[0, 0, 0], kp[0, 0, 1], kp[4, 0, 0]])
    v = np.stack([vp[3, 0, 0], vp[3, 0, 1], vp[0, 0, 0], vp[0, 0, 1], vp[4, 0, 0]])
    for t, n in ((0, 4), (1, 5)):
        for h in range(2):
            e = [np.exp(sum(q[t, h, c] * k[j, c] for c in range(4)) / 2.0) for j in range(n)]
            for c in range(4):
                assert abs(o[t, h, c] - sum(e[j] * v[j, c] for j in range(n)) / sum(e)) < 1e-12
            assert abs(lse[t, h] - np.log(sum(e))) < 1e-12
    assert np.isnan(o[2]).all()                     # a token of no sequence
    # nothing to see: zero and -inf
    o, lse, _, _ = po.attention(q, kp, vp, [0, 3], [2], table)
    assert (o[0] == 0).all() and (lse[0] == -np.inf).all() and np.isfinite(lse[1]).all()


def test_oracle_page_score_bounds_every_key():
    rng = np.random.default_rng(2)
    kp = rng.normal(size=(6, 1, 4, 8))
    q = rng.normal(size=(1, 3, 8))
    mn, mx = kp.min(2), kp.max(2)
    table = np.array([[5, 4, 3, 2, 1, 0]])
    pages, counts = po.select_pages(q, mn, mx, [0, 1], [24], table, 4, 2, 1, 1)
    assert counts[0, 0] == 4 and pages[0, 0, 0] == 0 and pages[0, 0, 3] == 5
    bound = [np.maximum(q[0] * mn[p, 0], q[0] * mx[p, 0]).sum() for p in table[0]]
    for j, p in enumerate(table[0]):
        assert (kp[p, 0] @ q[0].T).sum(1).max() <= bound[j] + 1e-12
    assert sorted(pages[0, 0, 1:3]) == sorted(sorted(range(1, 5), key=lambda j: -bound[j])[:2])
    # equal scores: the lowest pages
    one = np.ones_like(mn)
    pages, _ = po.select_pages(np.abs(q), one, one, [0, 1], [24], table, 4, 2, 1, 1)
    assert pages[0, 0].tolist() == [0, 1, 2, 5]
