"""Calls of qgemv_attn_shared with groups, shares and lengths of any kind, against the definition in 64 bits."""
from __future__ import annotations

import ctypes

import numpy as np

from gpu_common import D, dev, host, q, say, torch
from kv_common import BYTES, Cache, check_rows, held, parts64, scales64


def form_of(kv_type, n_seq, n_group, nq, nkv, hd, positions):
    """The kernels that take a call: by 16-column tiles, or by 128-column ones in three ways."""
    fn = ctypes.CDLL(q.LIB_PATH)["_ZN2qg11shared_formEiliiiil"]
    fn.restype = ctypes.c_int
    fn.argtypes = [ctypes.c_int, ctypes.c_int64, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int64]
    return ["16", "parted", "few", "whole"][fn(kv_type, n_seq, n_group, nq, nkv, hd, positions)]


def int32s(x):
    return torch.tensor([int(v) for v in x], dtype=torch.int32, device="cuda")


class Batch:
    """Sequences with dense rows K, V of each ([len][nkv][hd], what is shared written out in all of them), each in
    pages of its own."""

    def __init__(self, kv_type, K, V, nq, nkv, hd, page=16, seed=0, extra_entries=2, q_size=1.0,
                 scale=None):
        rng = np.random.default_rng([95, seed])
        self.kv_type, self.K, self.V, self.nq, self.nkv, self.hd = kv_type, K, V, nq, nkv, hd
        self.n, self.scale = len(K), hd ** -0.5 if scale is None else scale
        self.c = Cache(kv_type, K, V, page, nkv, hd, rng, extra_entries=extra_entries)
        self.x = (rng.standard_normal((self.n, nq * hd)) * q_size).astype(np.float32)
        self.q = dev(self.x)
        self.ws = D.attn_workspace(q.OP_ATTN_SHARED, self.n, nq, nkv, hd)

    def form(self, n_group):
        return form_of(self.kv_type, self.n, n_group, self.nq, self.nkv, self.hd, self.c.max_pages * self.c.page)

    def call(self, starts, share, lens, n_group=None, ws=None):
        """The outputs and the flag."""
        n_group = len(starts) - 1 if n_group is None else n_group
        say(f"shared type={self.kv_type} n={self.n} heads={self.nq}/{self.nkv}x{self.hd} groups={n_group} "
            f"starts={list(starts)[:6]} share={list(share)[:6]} lens={list(lens)[:6]} {self.form(n_group)}")
        o = torch.full((self.n, self.nq * self.hd), float("nan"), device="cuda")
        ws = self.ws if ws is None else ws
        q.qgemv_attn_shared(*self.c.args(), int32s(lens), self.n, int32s(starts), int32s(share), n_group, self.q,
                            self.nq * self.hd, self.nq, self.scale, o, ws)
        return host(o), q.qgemv_attn_error(ws)

    def check(self, got, seen, what="shared"):
        """seen: the positions that each row attends to, a number (so many from the first) or an array."""
        parts, n = [], []
        for b in range(self.n):
            at = np.arange(seen[b]) if np.ndim(seen[b]) == 0 else seen[b]
            k, v = self.K[b][at], self.V[b][at]
            dv = scales64(v, self.kv_type) if self.kv_type in BYTES and len(v) else np.ones(v.shape[:2])
            parts.append(parts64(self.x[b].reshape(self.nq, self.hd), held(k, self.kv_type), held(v, self.kv_type), dv,
                                 self.nkv, self.scale, len(at) - 1, self.kv_type))
            n.append(len(at))
        check_rows(got, parts, n, self.hd, self.kv_type, what)
