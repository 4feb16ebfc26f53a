"""Shared helpers of the attention-side tests: a paged cache built from dense K and V, the 64-bit
definitions of attention and routing, and the derived tolerances.

Attention tolerance, per output channel, with A = sum_t p_t |v_t|, S = max_t scale sum_d |q_d k_td|,
n positions and u = 2^-24 (half a step of f32): a score is off by at most (e + (hd + 4) u) S, e
being what the split of q leaves (two halves: f16 2^-22, bf16 2^-18); a relative error d of every
weight moves o by at most 2 d A; the weights' own split leaves e, exp and the scaling a few u, and
the sums of n products and of n weights at most n u each.  Together
    |o - ref| <= (2 (e + (hd + 4) u) S + 2 e + 16 u + 2 n u) A.
That holds for any order of the sums; the root of the mean square error against that of A is held
to 2^-16 as well (the terms' signs are random: bf16 leaves about 2^-18 times the few units of S),
which one rounding of q or of the weights to f16 (2^-12) would miss.
"""
from __future__ import annotations

import numpy as np

from gpu_common import q, torch

U = 2.0 ** -24
TORCH = {q.F16: torch.float16, q.BF16: torch.bfloat16}
LEFT = {q.F16: 2.0 ** -22, q.BF16: 2.0 ** -18}


def rounded(a, kv_type):
    """f32 values rounded to the cache's type (to nearest-even), as f32."""
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(TORCH[kv_type]).float().numpy()


class Paged:
    """A paged cache with dense K, V of each sequence ([len][nkv][hd], f32 values of the type):
    pages at random places of the pool, `fill` in every other place of it."""

    def __init__(self, kv_type, K, V, page, nkv, hd, rng, spare=3, extra_entries=2, fill=float("nan"),
                 page_stride=None, bad_entry=-1):
        self.kv_type, self.page, self.nkv, self.hd = kv_type, page, nkv, hd
        need = [-(-len(k) // page) for k in K]
        self.n_seq, self.n_pages = len(K), sum(need) + spare
        self.max_pages = max(need) + extra_entries
        block = nkv * page * hd
        self.page_stride = block if page_stride is None else page_stride
        kp = np.full((self.n_pages, nkv, page, hd), fill, dtype=np.float32)
        vp = np.full((self.n_pages, nkv, hd, page), fill, dtype=np.float32)
        table = np.full((self.n_seq, self.max_pages), bad_entry, dtype=np.int32)
        perm = rng.permutation(self.n_pages)
        at = 0
        for b, (k, v) in enumerate(zip(K, V)):
            for i in range(need[b]):
                pg = int(perm[at])
                at += 1
                table[b, i] = pg
                part = k[i * page:(i + 1) * page]
                kp[pg, :, :len(part)] = part.transpose(1, 0, 2)
                vp[pg, :, :, :len(part)] = v[i * page:(i + 1) * page].transpose(1, 2, 0)
        self.table_host = table
        self.table = torch.from_numpy(table).cuda()
        self.kv_len_host = np.array([len(k) for k in K], dtype=np.int32)
        self.kv_len = torch.from_numpy(self.kv_len_host).cuda()
        self.k, self.v = self._pool(kp, block), self._pool(vp, block)

    def _pool(self, a, block):
        t = torch.from_numpy(a.reshape(self.n_pages, block)).to(TORCH[self.kv_type])
        pool = torch.full((self.n_pages, self.page_stride), float("nan"), dtype=t.dtype)
        pool[:, :block] = t
        return pool.cuda()

    def args(self):
        return (self.kv_type, self.k, self.v, self.n_pages, self.page, self.page_stride, self.nkv,
                self.hd, self.table, self.max_pages)


def attention64(qr, K, V, nkv, scale, last):
    """One row's attention in f64: qr [nq][hd], K, V [len][nkv][hd], positions 0..last.  Returns o
    [nq][hd], A (same shape) and S [nq][1]."""
    nq, hd = qr.shape
    o, A, S = np.zeros((nq, hd)), np.zeros((nq, hd)), np.zeros((nq, 1))
    if last < 0:
        return o, A, S
    for h in range(nq):
        k = K[:last + 1, h // (nq // nkv)].astype(np.float64)
        v = V[:last + 1, h // (nq // nkv)].astype(np.float64)
        s = scale * (k @ qr[h].astype(np.float64))
        p = np.exp(s - s.max())
        p /= p.sum()
        o[h], A[h] = p @ v, p @ np.abs(v)
        S[h] = abs(scale) * (np.abs(k) @ np.abs(qr[h].astype(np.float64))).max()
    return o, A, S


def check_attention(got, ref, A, S, n, hd, kv_type, what):
    """got, ref, A [rows][nq * hd]; S [rows][nq]; n [rows] positions seen."""
    e = LEFT[kv_type]
    f = 2 * (e + (hd + 4) * U) * S + 2 * e + 16 * U + 2 * np.asarray(n, dtype=np.float64)[:, None] * U
    tol = np.repeat(f, hd, axis=1) * A
    err = np.abs(got.astype(np.float64) - ref)
    assert not np.isnan(got).any(), f"{what}: NaN"
    bad = err > tol
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.size} outside, worst "
                           f"{float((err / np.maximum(tol, 1e-300)).max()):.3g} of the tolerance")
    if A.any():
        rms = np.sqrt((err ** 2).mean()) / np.sqrt((A ** 2).mean())
        assert rms <= 2.0 ** -16, f"{what}: rms error {rms:.3g}"


def route64(z, score, bias, n_group, group_top, topk_group, topk, renorm, scale):
    """Routing by its definition in f64, one row after the other, with stable sorts."""
    z = np.asarray(z, dtype=np.float64)
    rows, n = z.shape
    ids, wts = np.zeros((rows, topk), np.int32), np.zeros((rows, topk))
    for r in range(rows):
        if score == q.SCORE_SIGMOID:
            s = 1.0 / (1.0 + np.exp(-z[r]))
        else:
            e = np.exp(z[r] - z[r].max())
            s = e / e.sum()
        c = s + (0.0 if bias is None else np.asarray(bias, dtype=np.float64))
        c = np.where(np.isnan(c), -np.inf, c)
        left = np.arange(n)
        if n_group > 1:
            g = -np.sort(-c.reshape(n_group, -1), axis=1)[:, :group_top].sum(axis=1)
            kept = np.sort(np.argsort(-g, kind="stable")[:topk_group])
            left = np.concatenate([np.arange(k * (n // n_group), (k + 1) * (n // n_group)) for k in kept])
        ids[r] = left[np.argsort(-c[left], kind="stable")[:topk]]
        w = s[ids[r]]
        if renorm:
            w = w / w.sum() if w.sum() != 0 else np.zeros_like(w)
        wts[r] = w * scale
    return ids, wts
