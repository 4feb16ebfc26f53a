"""Bounds that hold the attentions to the bits their operands carry, and an emulation of that arithmetic.

A scaled query and a probability enter the products as the sum of two f16 or three bf16 values, K and V as
stored, everything else is f32 (u = 2^-24 half a step of it).  In logarithms to the base 2 a score s is off by
a random error of several parts, given here as root mean squares:
  - the query's pieces: relative 2^-23 (f16: the second piece rounds at 2^-11 of a remainder of 2^-12; bf16:
    nothing) of the products' root of sum of squares, Q = scale log2 e sqrt(sum_d (q_d k_d)^2);
  - the f32 sums over head_dim and pieces and the factors before and after: a few u Q and u |s|;
  - s plus the reference's exponent, at most 16 in magnitude where the weight matters: 2^-21 / sqrt(3).
A weight then has ln 2 times that as its relative error, and from exp2 and its own two pieces 2^-23 / sqrt(3)
each.  For Q and |s| of a few units that makes less than 2^-21 (1 + Q') with Q' = Q ln 2, the same in natural
logarithms: at Q' = 1, ln 2 (2^-21 / sqrt(3) = 2.8e-7, 4 u Q = 3.4e-7) and 1e-7 together 3.3e-7 of the bound's
9.5e-7.  Two bf16 pieces leave 2^-18 of each query channel and of each weight at most, 2^-18 / sqrt(3) 0.75 =
1.65e-6 as a root mean square over a binade: 1.65e-6 sqrt(1 + Q'^2), 2.3e-6 at Q' = 1, outside; and one f16
piece 2^-12, far outside.

Independent errors d of the weights move o = sum p v / sum p by d sqrt(sum p^2 (v - o)^2), and the f32 sums and
the division by some u |o|; so the root of the mean square of (error) over that of
N = sqrt(sum p^2 (v - o)^2 + o^2) is held to 2^-21 (1 + Q').

Far below the largest weight the two f16 pieces end at the type's least step 2^-24: weights are held times
2^10 of the reference, which is no larger than the largest, so that what is lost there is at most half a step,
2^-25 / 2^10 = 2^-35 of the largest weight, for every position.
"""
from __future__ import annotations

import numpy as np

from gpu_common import q

U = 2.0 ** -24
F16_LOST = 2.0 ** -35               # of the largest weight, a position


def parts64(qr, K, V, nkv, scale, last):
    """One row in f64: o [nq][hd], N (same), Q' [nq], the weights over the largest [nq][last + 1]."""
    nq, hd = qr.shape
    o, N, Q, W = np.zeros((nq, hd)), np.zeros((nq, hd)), np.zeros(nq), np.zeros((nq, last + 1))
    for h in range(nq):
        k = K[:last + 1, h // (nq // nkv)].astype(np.float64)
        v = V[:last + 1, h // (nq // nkv)].astype(np.float64)
        x = qr[h].astype(np.float64)
        s = scale * (k @ x)
        W[h] = np.exp(s - s.max())
        p = W[h] / W[h].sum()
        o[h] = p @ v
        N[h] = np.sqrt((p ** 2) @ (v - o[h]) ** 2 + o[h] ** 2)
        Q[h] = abs(scale) * np.sqrt(((k ** 2) @ (x ** 2) * p).sum())       # where the weight is
    return o, N, Q, W


def rms_ratio(got, o, N):
    return float(np.sqrt(((got.astype(np.float64) - o) ** 2).mean()) / np.sqrt((N ** 2).mean()))


def rms_bound(Q):
    return 2.0 ** -21 * (1.0 + float(np.sqrt((np.asarray(Q) ** 2).mean())))


def pieces(a, kv_type, count):
    """f32 values as the sum of `count` values of the type, each rounded to nearest-even."""
    import torch
    dt = {q.F16: torch.float16, q.BF16: torch.bfloat16}[kv_type]
    left, out = torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)), []
    for _ in range(count):
        p = left.to(dt).float()
        out.append(p.numpy())
        left = left - p
    return out


def emulate(qr, K, V, scale, kv_type, q_pieces, p_pieces, lift):
    """One head's attention as the kernels compute it: qr [hd], K, V [n][hd]; weights held times 2^lift."""
    f = np.float32
    amax = np.abs(qr).max()
    sc = f(2.0) ** (14 - np.frexp(amax)[1]) if kv_type == q.F16 else f(1.0)
    s = np.zeros(len(K), f)
    for piece in reversed(pieces(qr.astype(f) * sc, kv_type, q_pieces)):
        for k0 in range(0, len(qr), 32):
            s = (s.astype(np.float64) + K[:, k0:k0 + 32].astype(np.float64) @ piece[k0:k0 + 32]).astype(f)
    s = s * (f(scale) * f(np.log2(np.e)) / sc)
    p = np.exp2((s + (f(lift) - s.max())).astype(np.float64)).astype(f)
    o = np.zeros(V.shape[1], f)
    for t0 in range(0, len(K), 32):
        for piece in reversed(pieces(p[t0:t0 + 32], kv_type, p_pieces)):
            o = (o.astype(np.float64) + piece.astype(np.float64) @ V[t0:t0 + 32].astype(np.float64)).astype(f)
    l = f(0.0)
    for t0 in range(0, len(K), 32):
        l = l + p[t0:t0 + 32].sum(dtype=f)
    return o / l


def tail_case(rng, n, hd, bits, kv_type, equal):
    """One position with the whole weight and no value, n - 1 others 2^-bits of its weight or less: the
    output is made of what is left of the small weights.  Returns q [hd], K, V [n][hd] for scale 1."""
    K = np.zeros((n, hd), np.float32)
    V = rng.standard_normal((n, hd)).astype(np.float32)
    x = np.zeros(hd, np.float32)
    x[0] = 1.0
    step = 2.0 ** -6
    K[1:, 0] = -np.round((bits * np.log(2.0) + (0.0 if equal else 1.0) * rng.uniform(0, 2, n - 1)) / step) * step
    V[0] = 0.0
    import torch
    dt = {q.F16: torch.float16, q.BF16: torch.bfloat16}[kv_type]
    r = lambda a: torch.from_numpy(a).to(dt).float().numpy()
    return x, r(K), r(V)


def tail_tolerance(W, V, hd, kv_type):
    """Of one head of a tail_case: W the weights over the largest, V [n][hd]; elementwise.  Scores up to S
    (all in one channel: the query's pieces are exact, one product) and f32 work as in attn_common, with the
    position's own lost bits."""
    n, p = len(W), W / W.sum()
    S = float(-np.log(W).min())
    A = p @ np.abs(V.astype(np.float64))
    rel = 2 * (2.0 ** -22 + 8 * U) * S + 2 * 2.0 ** -22 + 2.0 ** -20 + 2 * n * U
    lost = F16_LOST if kv_type == q.F16 else 0.0
    return rel * A + lost * np.abs(V.astype(np.float64)).sum(axis=0) / W.sum()


def dominant_case(rng, n, hd, kv_type):
    """A first position with about 90 % of the weight and a value a hundredth of the others', as a language
    model's attention has it.  Returns q [hd], K, V [n][hd] for scale hd^-1/2."""
    import torch
    dt = {q.F16: torch.float16, q.BF16: torch.bfloat16}[kv_type]
    x = rng.standard_normal(hd).astype(np.float32)
    K, V = rng.standard_normal((n, hd)).astype(np.float32), rng.standard_normal((n, hd)).astype(np.float32)
    s = K[1:].astype(np.float64) @ x * hd ** -0.5
    K[0] = x / (x @ x) * (np.log(9.0) + np.log(np.exp(s).sum())) * hd ** 0.5
    V[0] *= 0.01
    r = lambda a: torch.from_numpy(a).to(dt).float().numpy()
    return x, r(K), r(V)
