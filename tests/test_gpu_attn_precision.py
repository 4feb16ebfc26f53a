"""The attentions held to the bits that their operands carry (attn_precision), in the three kernels: one token,
16-column and 128-column tiles; and values, keys and scales near the ends of what the types hold."""
import numpy as np
import pytest

from gpu_common import dev, host, require_gpu, say, torch

import dequant_gemv_q4_amd as q
from dequant_gemv_q4_amd import device as D
from attn_common import Paged, attention64, check_attention, rounded
from attn_precision import dominant_case, parts64, rms_bound, rms_ratio, tail_case, tail_tolerance

pytestmark = pytest.mark.gpu

TYPES = [q.F16, q.BF16]
# rows of one sequence: single token, a 16-column tile's, 128-column tiles' (with a group of 4 or more)
ROWS = [0, 8, 130]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _run(kv_type, nq, nkv, hd, page, x, K, V, rows, scale):
    """One sequence of K, V [n][nkv][hd] and its last rows x [rows or 1][nq][hd]."""
    m = max(rows, 1)
    assert x.shape == (m, nq, hd) and (rows < 100 or rows * (nq // nkv) > 384)
    c = Paged(kv_type, [K], [V], page, nkv, hd, np.random.default_rng(64), extra_entries=1040 // page)
    xd, o = dev(np.ascontiguousarray(x.reshape(m, nq * hd))), torch.full((m, nq * hd), float("nan"), device="cuda")
    ws = D.attn_workspace(q.OP_ATTN_PROMPT, 1, nq, nkv, hd)
    if rows:
        q.qgemv_attn_prompt(*c.args(), torch.tensor([0, m], dtype=torch.int32, device="cuda"), c.kv_len, 1, xd,
                            nq * hd, m, nq, scale, o, ws)
    else:
        q.qgemv_attn(*c.args(), c.kv_len, 1, xd, nq * hd, nq, scale, o, ws)
    return host(o).reshape(m, nq, hd)


@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("kv_type", TYPES)
@pytest.mark.parametrize("nq,nkv,hd,n,spread", [(8, 2, 64, 300, 1.0), (8, 2, 128, 300, 1.5), (4, 1, 256, 300, 1.0),
                                                (8, 2, 128, 300, 4.0), (4, 1, 192, 1500, 1.0), (5, 1, 96, 700, 1.0)])
def test_normal_inputs(kv_type, nq, nkv, hd, n, spread, rows):
    rng = np.random.default_rng([65, hd, rows])
    m = max(rows, 1)
    got, o, N, Q = [], [], [], []
    for _ in range(4 if m < 16 else 1):
        x = (rng.standard_normal((m, nq, hd)) * spread).astype(np.float32)
        K, V = (rounded(rng.standard_normal((n, nkv, hd)), kv_type) for _ in range(2))
        got.append(_run(kv_type, nq, nkv, hd, 16, x, K, V, rows, hd ** -0.5))
        for r in range(m):
            a, b, c, _ = parts64(x[r], K, V, nkv, hd ** -0.5, n - m + r)
            o.append(a)
            N.append(b)
            Q.append(c)
    err, bound = rms_ratio(np.concatenate(got), np.stack(o), np.stack(N)), rms_bound(np.stack(Q))
    say(f"precision type={kv_type} hd={hd} n={n} spread={spread} rows={rows}: {err:.3g} of {bound:.3g}")
    assert err <= bound


@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("kv_type", TYPES)
@pytest.mark.parametrize("equal", [False, True])
@pytest.mark.parametrize("bits", [12, 20, 24, 27])
def test_small_weights_beside_a_large_one(kv_type, equal, bits, rows):
    hd, nq, m = 64, 4, max(rows, 1)
    n = 129 + m
    rng = np.random.default_rng([66, bits])
    worst = 0.0
    for _ in range(6):
        x, K, V = tail_case(rng, n, hd, bits + rng.uniform(0, 1), kv_type, equal)
        got = _run(kv_type, nq, 1, hd, 16, np.broadcast_to(x, (m, nq, hd)).copy(), K[:, None], V[:, None], rows, 1.0)
        for r in range(0, m, 7):
            last = n - m + r
            o, _, _, W = parts64(x[None], K[:, None], V[:, None], 1, 1.0, last)
            tol = tail_tolerance(W[0], V[:last + 1], hd, kv_type)
            worst = max(worst, float((np.abs(got[r] - o[0]) / tol).max()))
    say(f"small weights type={kv_type} bits={bits} equal={equal} rows={rows}: {worst:.3g} of the tolerance")
    assert worst <= 1.0


@pytest.mark.parametrize("kv_type", TYPES)
def test_a_dominant_first_position(kv_type):
    """A whole prompt of 8192 rows, whose tiles are not split: one reference covers all positions."""
    hd, nq, n = 64, 8, 8192
    rng = np.random.default_rng(67)
    x0, K, V = dominant_case(rng, n, hd, kv_type)
    x = (x0 + 0.02 * rng.standard_normal((n, nq, hd))).astype(np.float32)
    got = _run(kv_type, nq, 1, hd, 64, x, K[:, None], V[:, None], n, hd ** -0.5)
    at = list(range(4000, n, 131)) + [n - 1]
    o, N, Q, W = zip(*(parts64(x[r], K[:, None], V[:, None], 1, hd ** -0.5, r) for r in at))
    assert all(0.8 < w[0, 0] / w[0].sum() < 0.99 for w in W)
    err, bound = rms_ratio(got[at], np.stack(o), np.stack(N)), rms_bound(np.stack(Q))
    say(f"dominant position type={kv_type}: {err:.3g} of {bound:.3g}")
    assert err <= bound
    for rows in ROWS[:2]:
        m = max(rows, 1)
        got = _run(kv_type, nq, 1, hd, 64, x[n - m:], K[:, None], V[:, None], rows, hd ** -0.5)
        o, N, Q, _ = zip(*(parts64(x[r], K[:, None], V[:, None], 1, hd ** -0.5, r) for r in range(n - m, n)))
        assert rms_ratio(got, np.stack(o), np.stack(N)) <= rms_bound(np.stack(Q))
