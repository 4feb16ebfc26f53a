"""Shared helpers of the tests of the 8-bit cache, the fused QKV append and shared prefixes: quantisation
by its definition, a paged cache of any type built from dense rows, and the derived tolerances.

A cached value is exact (scale * code, or an f16 / bf16 value), so the tolerance of attn_common holds for
the 8-bit types with f16's two pieces, and with the roundings that the scales add: of a score one (d^K),
of a weight one (d^V), of a row whose positions are read in two parts a few of the join's factors:
    |o - ref| <= (2 (e + (hd + 6) u) S + 2 e + 24 u + 2 n u) A.
The product of a weight and its scale is held in two f16 pieces whose least step is 2^-24, times 2^10 of
the largest weight times the largest scale that the row sees: 2^-35 of that product times |code| is lost at
most a position, B = n 2^-35 max_t d_t max |code| / (sum of the weights over the largest, at least 1).
"""
from __future__ import annotations

import numpy as np

from gpu_common import q, torch
from attn_common import TORCH, U

LEFT = {q.F16: 2.0 ** -22, q.BF16: 2.0 ** -18, q.I8: 2.0 ** -22, q.F8: 2.0 ** -22}
NAMES = {q.F16: "f16", q.BF16: "bf16", q.I8: "i8", q.F8: "f8"}
CODES = {q.I8: 127.0, q.F8: 448.0}
ALL = [q.F16, q.BF16, q.I8, q.F8]
BYTES = [q.I8, q.F8]


def scales64(x, kv_type):
    """Scales of rows (the last axis) by their definition: f64 arithmetic on f32 or f64 values."""
    amax = np.abs(np.asarray(x, dtype=np.float64)).max(axis=-1)
    if kv_type == q.I8:
        return np.maximum((amax / 127).astype(np.float32), np.float32(2.0 ** -126))
    m, e = np.frexp(amax)
    k = np.where(amax == 0, -126, np.maximum(e - 9 + (m > 0.875), -126))
    return np.ldexp(np.float64(1.0), k).astype(np.float32)


def codes64(x, d, kv_type):
    """Codes, as the numbers they are, and how far each quotient is from the nearest border between two
    codes, relative to the code's step."""
    y = np.asarray(x, dtype=np.float64) / d[..., None].astype(np.float64)
    if kv_type == q.I8:
        step = np.ones_like(y)
    else:
        _, e = np.frexp(y)
        step = np.ldexp(1.0, np.maximum(e - 4, -9))       # e4m3: three bits behind the first, 2^-9 at least
    n = np.rint(y / step)
    return n * step, 0.5 - np.abs(y / step - n)


def quantised(x, kv_type):
    """(codes, scales); a row that is not finite has scale NaN and codes 0."""
    x = np.asarray(x)
    fine = np.isfinite(x).all(axis=-1)
    safe = np.where(fine[..., None], x, 0)
    d = scales64(safe, kv_type)
    c, _ = codes64(safe, d, kv_type)
    return c, np.where(fine, d, np.float32("nan"))


def held(x, kv_type):
    """What a cache of the type holds of f32 or f64 rows, as f64: one rounding."""
    x = np.asarray(x)
    if kv_type in BYTES:
        c, d = quantised(x, kv_type)
        return c * d[..., None].astype(np.float64)
    if x.dtype == np.float64:                             # (of values within the type's range)
        bits, least = (11, -13) if kv_type == q.F16 else (8, -125)
        step = np.ldexp(1.0, np.maximum(np.frexp(x)[1], least) - bits)
        return np.rint(x / step) * step
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(TORCH[kv_type]).double().numpy()


def as_bytes(codes, kv_type):
    if kv_type == q.I8:
        return codes.astype(np.int8).view(np.uint8)
    return torch.from_numpy(codes.astype(np.float32)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()


class Cache:
    """A paged cache of any type with dense rows K, V of each sequence ([len][nkv][hd], f32): pages at
    random places of the pool; every other place of it holds NaN (8-bit: NaN scales and, of f8, NaN codes).
    tables: entries that sequences share, {(sequence, entry): (other, entry)}."""

    def __init__(self, kv_type, K, V, page, nkv, hd, rng, spare=3, extra_entries=2, bad_entry=-1, gap=0,
                 tables=None):
        self.kv_type, self.page, self.nkv, self.hd = kv_type, page, nkv, hd
        bytes_ = kv_type in BYTES
        self.block = page * (hd + 4 if bytes_ else hd)
        self.page_stride = nkv * self.block + gap
        need = [-(-len(k) // page) for k in K]
        tables = tables or {}
        self.n_seq, self.n_pages = len(K), sum(need) + spare
        self.max_pages = max(need + [0]) + extra_entries
        table = np.full((self.n_seq, self.max_pages), bad_entry, dtype=np.int32)
        perm = rng.permutation(self.n_pages)
        if bytes_:
            k = np.full((self.n_pages, self.page_stride), 0x7F, dtype=np.uint8)   # 0x7F7F7F7F f32: 3.4e38
            v = k.copy()
            for a in (k, v):
                for h in range(nkv):
                    at = h * self.block + page * hd
                    a[:, at:at + 4 * page] = np.frombuffer(np.float32("nan").tobytes() * page, np.uint8)
        else:
            k = np.full((self.n_pages, self.page_stride), np.nan, dtype=np.float32)
            v = k.copy()
        at = 0
        for b in range(self.n_seq):
            for i in range(need[b]):
                if (b, i) in tables:
                    table[b, i] = table[tables[b, i]]
                    continue
                pg = table[b, i] = int(perm[at])
                at += 1
                for pool, rows, turned in ((k, K[b], False), (v, V[b], True)):
                    part = rows[i * page:(i + 1) * page]
                    if not bytes_:
                        x = np.full((nkv, page, hd), np.nan, np.float32)
                        x[:, :len(part)] = part.transpose(1, 0, 2)
                        pool[pg, :nkv * self.block] = (x.transpose(0, 2, 1) if turned else x).reshape(-1)
                        continue
                    codes, d = quantised(part.transpose(1, 0, 2), kv_type)       # [nkv][n][hd]
                    raw = np.full((nkv, page, hd), 0x7F, np.uint8)
                    raw[:, :len(part)] = as_bytes(codes, kv_type)
                    raw = raw.transpose(0, 2, 1) if turned else raw
                    scale = np.full((nkv, page), np.nan, np.float32)
                    scale[:, :len(part)] = d
                    both = np.concatenate([raw.reshape(nkv, -1), scale.view(np.uint8).reshape(nkv, -1)], 1)
                    pool[pg, :nkv * self.block] = both.reshape(-1)
        self.table_host = table
        self.table = torch.from_numpy(table).cuda()
        self.kv_len_host = np.array([len(x) for x in K], dtype=np.int32)
        self.kv_len = torch.from_numpy(self.kv_len_host).cuda()
        self.k, self.v = (torch.from_numpy(a) if bytes_ else torch.from_numpy(a).to(TORCH[kv_type])
                          for a in (k, v))
        self.k, self.v = self.k.cuda(), self.v.cuda()

    def args(self):
        return (self.kv_type, self.k, self.v, self.n_pages, self.page, self.page_stride, self.nkv,
                self.hd, self.table, self.max_pages)

    def read(self, pool, page, head, slot, turned):
        """Code (or value) and scale of position `slot` of a page's head in a copy of a pool."""
        blk = pool[page, head * self.block:(head + 1) * self.block]
        n = self.page * self.hd
        if self.kv_type in BYTES:
            dt = torch.int8 if self.kv_type == q.I8 else torch.float8_e4m3fn
            x = torch.from_numpy(blk[:n].copy()).view(dt).double().numpy()
            d = blk[n:].copy().view(np.float32)[slot]
        else:
            x, d = blk[:n], None
        x = x.reshape(self.hd, self.page).T if turned else x.reshape(self.page, self.hd)
        return x[slot], d


def parts64(qr, K, V, dV, nkv, scale, last, kv_type):
    """One row's attention in f64: qr [nq][hd], K, V [len][nkv][hd] as the cache holds them, dV [len][nkv] the
    scales of V, positions 0..last.  Returns o and A [nq][hd], S and B [nq][1] of the module's text."""
    nq, hd = qr.shape
    o, A, S, B = np.zeros((nq, hd)), np.zeros((nq, hd)), np.zeros((nq, 1)), np.zeros((nq, 1))
    if last < 0:
        return o, A, S, B
    n, g = last + 1, nq // nkv
    for h in range(nkv):
        rows = slice(h * g, (h + 1) * g)
        x = qr[rows].astype(np.float64)
        k, v = K[:n, h].astype(np.float64), V[:n, h].astype(np.float64)
        s = scale * (x @ k.T)
        w = np.exp(s - s.max(axis=1, keepdims=True))
        total = w.sum(axis=1, keepdims=True)
        p = w / total
        o[rows], A[rows] = p @ v, p @ np.abs(v)
        S[rows] = abs(scale) * (np.abs(x) @ np.abs(k).T).max(axis=1, keepdims=True)
        if kv_type in BYTES:
            B[rows] = n * 2.0 ** -35 * dV[:n, h].max() * CODES[kv_type] / total
    return o, A, S, B


def check_rows(got, parts, n, hd, kv_type, what):
    """got [rows][nq * hd]; parts of each row (o, A, S, B); n positions seen of each."""
    ref, A, S, B = (np.stack([p[i].reshape(-1) for p in parts]) for i in range(4))
    e = LEFT[kv_type]
    f = 2 * (e + (hd + 6) * U) * S + 2 * e + 24 * U + 2 * np.asarray(n, dtype=np.float64)[:, None] * U
    tol = np.repeat(f, hd, axis=1) * A + np.repeat(B, hd, axis=1)
    err = np.abs(got.astype(np.float64) - ref)
    assert not np.isnan(got).any(), f"{what}: NaN"
    bad = err > tol
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.size} outside, worst "
                           f"{float((err / np.maximum(tol, 1e-300)).max()):.3g} of the tolerance")
    for r, seen in enumerate(n):
        if seen <= 0:
            assert not got[r].any(), f"{what}: row {r} sees nothing"
    if A.any():
        rms = np.sqrt((err ** 2).mean()) / np.sqrt((A ** 2).mean())
        assert rms <= 2.0 ** -16, f"{what}: rms error {rms:.3g}"
