"""Batches of the paged-cache tests, and their tolerances.

A Batch holds a page pool in which every row that no sequence owns is NaN (the
page tails, the unused pages) and a page table whose entries behind a
sequence's last page are wild numbers: none of it may show in a result.
"""
import numpy as np
import torch

from oracle import paged_oracle as po

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}      # half a step, relative
TINY = {torch.bfloat16: 0.0, torch.float16: 2.0 ** -25}         # half the smallest fp16


def f64(t):
    return t.detach().double().cpu().numpy()


class Batch:
    def __init__(self, q_lens, kv_lens, Hq, Hkv, d, ps, dtype, seed=0, extra=0, scale=1.0):
        g = torch.Generator().manual_seed(seed)
        self.q_lens, self.kv_lens, self.ps, self.dtype = q_lens, kv_lens, ps, dtype
        self.Hq, self.Hkv, self.d = Hq, Hkv, d
        self.cu = [0]
        for x in q_lens:
            self.cu.append(self.cu[-1] + x)
        self.n = self.cu[-1] + extra
        need = [(x + ps - 1) // ps for x in kv_lens]
        self.n_pages = sum(need) + 2
        maxp = max(max(need), 1) + 2
        perm = torch.randperm(self.n_pages, generator=g)
        table = torch.full((len(kv_lens), maxp), 2 ** 30, dtype=torch.int32)
        k = torch.full((self.n_pages, Hkv, ps, d), float("nan"))
        v = torch.full((self.n_pages, Hkv, ps, d), float("nan"))
        at = 0
        for s, m in enumerate(need):
            ids = perm[at:at + m]
            table[s, :m] = ids.int()
            at += m
            for i, p in enumerate(ids):
                r = min(ps, kv_lens[s] - i * ps)
                k[p, :, :r] = torch.randn(Hkv, r, d, generator=g) * scale
                v[p, :, :r] = torch.randn(Hkv, r, d, generator=g)
        self.table_host = table
        self.table = table.cuda()
        self.k, self.v = k.to(dtype).cuda(), v.to(dtype).cuda()
        self.q = torch.randn(max(self.n, 1), Hq, d, generator=g)[:self.n].to(dtype).cuda()
        self.cu_q = torch.tensor(self.cu, dtype=torch.int32, device="cuda")
        self.lens = torch.tensor(kv_lens, dtype=torch.int32, device="cuda")
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    @property
    def max_q(self):
        return max(max(self.q_lens), 1)

    def oracle(self, pages=None, counts=None):
        return po.attention(f64(self.q), f64(self.k), f64(self.v), self.cu, self.kv_lens,
                            self.table_host.numpy(), pages, counts)


def check_attention(o, lse, ref, dtype, d, p_round=0.0):
    """Outputs against the oracle's (o, lse, sum p|v|, largest sum |q k|/sqrt d).

    A score is a sum of d exact products; with each addition off by at most
    2^-23 of the running sum of magnitudes (truncating adders included) it is
    off by e_s = d 2^-23 max_j sum|q k|/sqrt(d).  2^x is good to 2^-21, and the
    weight's exponent s log2e - m rounds twice, 2^-23 of a magnitude of at most
    max|s| log2e <= 2 e_s 2^23 / d: together e_w = 3 e_s + 2^-20.  Numerator and
    denominator each carry it, P's rounding (p_round) only the numerator:
      |o - O| <= half a step of the output + (2 e_w + p_round + 2^-18) sum p|v|
    with 2^-18 for the additions over the keys (fp32, rescaled at most once a
    tile); |lse - L| <= 2 e_w + a rounding of it, 2^-22 |L|.
    """
    O, L, av, aq = ref
    live = ~np.isnan(L)
    o, lse = f64(o)[live], f64(lse)[live]
    O, L, av, aq = O[live], L[live], av[live], aq[live]
    empty = np.isneginf(L)
    assert (o[empty] == 0).all() and np.isneginf(lse[empty]).all()
    O, L, av, aq, o, lse = (x[~empty] for x in (O, L, av, aq, o, lse))
    if L.size == 0:
        return
    assert np.isfinite(o).all() and np.isfinite(lse).all()
    e_w = 3 * d * 2.0 ** -23 * aq + 2.0 ** -20
    delta = (2 * e_w + p_round + 2.0 ** -18)[..., None] * av
    err = np.abs(o - O) - (U[dtype] * (np.abs(O) + delta) + delta + TINY[dtype])
    assert err.max() <= 0, f"o off by {err.max():.3e} beyond its bound"
    el = np.abs(lse - L) - (2 * e_w + 2.0 ** -22 * np.abs(L))
    assert el.max() <= 0, f"lse off by {el.max():.3e} beyond its bound"
