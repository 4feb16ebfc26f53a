"""The precision bounds of attn_precision tell the operands' bits apart: the emulated arithmetic stays
within them, and one with a piece left out, or with weights lifted less, does not (no GPU)."""
import numpy as np
import pytest

import dequant_gemv_q4_amd as q
from attn_common import rounded
from attn_precision import dominant_case, emulate, parts64, rms_bound, rms_ratio, tail_case, tail_tolerance

LIFT = {q.F16: 10, q.BF16: -7}
PIECES = {q.F16: 2, q.BF16: 3}


def _rms(kv_type, hd, spread, q_pieces, p_pieces, heads=24, n=300):
    rng = np.random.default_rng([61, hd])
    got, ref, N, Q = [], [], [], []
    for _ in range(heads):
        x = (rng.standard_normal(hd) * spread).astype(np.float32)
        K, V = rounded(rng.standard_normal((n, hd)), kv_type), rounded(rng.standard_normal((n, hd)), kv_type)
        got.append(emulate(x, K, V, hd ** -0.5, kv_type, q_pieces, p_pieces, LIFT[kv_type]))
        o, w, s, _ = parts64(x[None], K[:, None], V[:, None], 1, hd ** -0.5, n - 1)
        ref.append(o[0])
        N.append(w[0])
        Q.append(s[0])
    return rms_ratio(np.stack(got), np.stack(ref), np.stack(N)), rms_bound(Q)


@pytest.mark.parametrize("kv_type", [q.F16, q.BF16])
@pytest.mark.parametrize("hd,spread", [(64, 1.0), (128, 1.5), (256, 1.0), (128, 4.0)])
def test_bound_holds_for_all_pieces_and_for_no_fewer(kv_type, hd, spread):
    full = PIECES[kv_type]
    err, bound = _rms(kv_type, hd, spread, full, full)
    assert err <= bound, (err, bound)
    fewer = [(full - 1, full), (full - 1, full - 1)]
    if spread <= 1.0:                                  # the bound grows with the scores, a weight's piece does not
        fewer.append((full, full - 1))
    for a, b in fewer:
        err, bound = _rms(kv_type, hd, spread, a, b)
        assert err > bound, (a, b, err, bound)


@pytest.mark.parametrize("kv_type", [q.F16, q.BF16])
@pytest.mark.parametrize("equal", [False, True])
@pytest.mark.parametrize("bits", [12, 20, 24, 27])
def test_small_weights_keep_their_bits_beside_a_large_one(kv_type, equal, bits):
    n, hd = 130, 64
    rng = np.random.default_rng([62, bits])
    worst = {LIFT[kv_type]: 0.0, 6: 0.0}
    for _ in range(12):
        x, K, V = tail_case(rng, n, hd, bits + rng.uniform(0, 1), kv_type, equal)
        o, _, _, W = parts64(x[None], K[:, None], V[:, None], 1, 1.0, n - 1)
        tol = tail_tolerance(W[0], V, hd, kv_type)
        for lift in worst:
            got = emulate(x, K, V, 1.0, kv_type, PIECES[kv_type], PIECES[kv_type], lift)
            worst[lift] = max(worst[lift], float((np.abs(got - o[0]) / tol).max()))
    assert worst[LIFT[kv_type]] <= 1.0, worst
    if kv_type == q.F16 and bits >= 20:
        assert worst[6] > 1.0, worst                  # half a step of 2^-31 shows


@pytest.mark.parametrize("kv_type", [q.F16, q.BF16])
@pytest.mark.parametrize("n", [1500, 8192])
def test_a_dominant_first_position(kv_type, n):
    hd, rng = 64, np.random.default_rng([63, n])
    got, ref, N, Q = {LIFT[kv_type]: [], 6: []}, [], [], []
    for _ in range(8):
        x, K, V = dominant_case(rng, n, hd, kv_type)
        o, w, s, W = parts64(x[None], K[:, None], V[:, None], 1, hd ** -0.5, n - 1)
        assert 0.85 < W[0, 0] / W[0].sum() < 0.95
        ref.append(o[0])
        N.append(w[0])
        Q.append(s[0])
        for lift, g in got.items():
            g.append(emulate(x, K, V, hd ** -0.5, kv_type, PIECES[kv_type], PIECES[kv_type], lift))
    err = {lift: rms_ratio(np.stack(g), np.stack(ref), np.stack(N)) for lift, g in got.items()}
    assert err[LIFT[kv_type]] <= rms_bound(Q), (err, rms_bound(Q))
    if kv_type == q.F16 and n > 8000:
        assert err[6] > rms_bound(Q), (err, rms_bound(Q))
