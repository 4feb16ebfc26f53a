"""Comparison of attention outputs some of which the definition leaves without a value: a query head of a
row that sees a NaN or infinite score has to come out non-finite in every channel, any other one within
the tolerance of attn_common."""
from __future__ import annotations

import numpy as np

from attn_common import attention64, check_attention


def attention64_rows(x, start, seqs, K, V, nkv, scale):
    """The rows of sequences (new rows, positions with them): reference, A [rows][nq][hd], S [rows][nq],
    positions seen [rows].  x [rows][nq][hd]."""
    ref, A, S, seen = [], [], [], []
    with np.errstate(all="ignore"):
        for b, (a, n) in enumerate(seqs):
            for i in range(a):
                o, w, s = attention64(x[start[b] + i], K[b], V[b], nkv, scale, n - a + i)
                ref.append(o)
                A.append(w)
                S.append(s[:, 0])
                seen.append(max(0, n - a + i + 1))
    return np.stack(ref), np.stack(A), np.stack(S), np.array(seen)


def check_finite_where_defined(got, ref, A, S, seen, kv_type, what):
    """got, ref, A [rows][nq][hd]."""
    got = got.reshape(ref.shape)
    rows, nq, hd = ref.shape
    lost = ~np.isfinite(ref)
    assert (~np.isfinite(got[lost])).all(), (f"{what}: {int(np.isfinite(got[lost]).sum())} of {int(lost.sum())} "
                                             f"outputs without a value came out finite")
    keep = ~lost.any(axis=2)
    n = np.repeat(np.asarray(seen)[:, None], nq, axis=1)
    if keep.any():
        check_attention(got[keep], ref[keep], A[keep], S[keep][:, None], n[keep], hd, kv_type, what)
    return int(lost.any(axis=2).sum())
