"""Scores without a value (NaN, or an infinite one) in the attentions: they may not vanish where they are all
that a wave, a chunk or a tile's part sees, nor where such a part's weight in the whole is 0, and they may
not reach a row or a head that does not see them."""
import numpy as np
import pytest

from gpu_common import dev, host, require_gpu, say, torch

import dequant_gemv_q4_amd as q
from dequant_gemv_q4_amd import device as D
from attn_common import Paged, rounded
from attn_nonfinite import attention64_rows, check_finite_where_defined

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _run(kv_type, nq, nkv, hd, page, seqs, x, K, V, decode, entries=2, scale=None):
    """x [rows][nq][hd]; decode: one row a sequence through qgemv_attn."""
    scale = hd ** -0.5 if scale is None else scale
    rng = np.random.default_rng(55)
    c = Paged(kv_type, K, V, page, nkv, hd, rng, extra_entries=entries)
    start = np.concatenate([[0], np.cumsum([a for a, _ in seqs])]).astype(np.int32)
    rows, n = int(start[-1]), len(seqs)
    xd = dev(np.ascontiguousarray(x.reshape(rows, nq * hd).astype(np.float32)))
    o = torch.full((rows, nq * hd), 77.0, device="cuda")
    ws = D.attn_workspace(q.OP_ATTN_PROMPT, n, nq, nkv, hd)
    kv = dev(np.array([b for _, b in seqs], np.int32))
    if decode:
        q.qgemv_attn(*c.args(), kv, n, xd, nq * hd, nq, scale, o, ws)
    else:
        q.qgemv_attn_prompt(*c.args(), dev(start), kv, n, xd, nq * hd, rows, nq, scale, o, ws)
    got = host(o)
    assert q.qgemv_attn_error(ws) == 0
    lost = check_finite_where_defined(got, *attention64_rows(x.astype(np.float32), start, seqs, K, V, nkv, scale),
                                      kv_type, f"decode={decode} {seqs[:4]}")
    say(f"nonfinite type={kv_type} hd={hd} decode={decode} seqs={seqs[:4]}: {lost} heads of rows without a value")
    return lost


def _draw(seed, lens, nq, nkv, hd, kv_type, rows):
    rng = np.random.default_rng([56, seed])
    K = [rounded(rng.standard_normal((max(0, n), nkv, hd)), kv_type) for n in lens]
    V = [rounded(rng.standard_normal((max(0, n), nkv, hd)), kv_type) for n in lens]
    return rng.standard_normal((rows, nq, hd)).astype(np.float32), K, V


TYPES = [q.F16, q.BF16]


@pytest.mark.parametrize("decode", [True, False])
@pytest.mark.parametrize("kv_type", TYPES)
@pytest.mark.parametrize("nq,nkv,hd", [(12, 2, 128), (3, 1, 64), (20, 1, 96), (4, 2, 256)])
def test_a_nan_key_that_a_wave_or_a_chunk_sees_alone(kv_type, nq, nkv, hd, decode):
    """Lengths of which the last position starts a wave's step or a chunk (513: the third of three)."""
    lens = [1, 33, 65, 97, 129, 40, 513, 2049, 0]
    x, K, V = _draw(hd, lens, nq, nkv, hd, kv_type, len(lens))
    for b, n in enumerate(lens):
        if n and n != 40:
            K[b][n - 1, 0, hd // 2] = np.nan
    lost = _run(kv_type, nq, nkv, hd, 16, [(1, n) for n in lens], x, K, V, decode)
    assert lost == 7 * (nq // nkv)
    x, K, V = _draw(hd + 1, [513], nq, nkv, hd, kv_type, 1)              # one sequence: in chunks
    K[0][512, nkv - 1, 1] = np.nan
    assert _run(kv_type, nq, nkv, hd, 16, [(1, 513)], x, K, V, decode) == nq // nkv


@pytest.mark.parametrize("decode", [True, False])
@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
@pytest.mark.parametrize("kv_type", TYPES)
def test_a_query_without_a_value(kv_type, bad, decode):
    """One head of one row NaN or infinite in one channel (or all), at short, long and no cache."""
    nq, nkv, hd = 12, 2, 128
    lens = [1, 32, 300, 3000, 0, 70, 9000]
    x, K, V = _draw(3, lens, nq, nkv, hd, kv_type, len(lens))
    x[0, 4, :], x[1, 0, 7], x[2, 11, :], x[3, 6, 100], x[4, 2, :], x[6, 1, :] = bad, bad, bad, bad, bad, bad
    lost = _run(kv_type, nq, nkv, hd, 32, [(1, n) for n in lens], x, K, V, decode)
    assert lost == 5


@pytest.mark.parametrize("kv_type", TYPES)
@pytest.mark.parametrize("nq,nkv,hd,seqs,entries", [
    (8, 2, 64, [(40, 40), (30, 90), (5, 3)], 2),                            # 16 columns a tile
    (8, 1, 128, [(3, 4000)], 2),                                            # split over the length
    (5, 1, 96, [(200, 200), (190, 700)], 70),                               # 128 columns, whole
    (8, 1, 128, [(61, 5000)], 2), (4, 1, 256, [(100, 2500)], 2),            # split, joined by a second launch
    (64, 4, 64, [(40, 6000), (300, 300), (250, 250), (400, 420), (330, 330), (100, 100)], 2),  # a few split
])
def test_prompt_queries_without_a_value(kv_type, nq, nkv, hd, seqs, entries):
    rows = sum(a for a, _ in seqs)
    x, K, V = _draw(4, [n for _, n in seqs], nq, nkv, hd, kv_type, rows)
    rng = np.random.default_rng(57)
    for r in rng.integers(0, rows, 12):
        x[r, rng.integers(0, nq), rng.integers(0, hd)] = rng.choice([np.nan, np.inf, -np.inf])
    x[1, 0, :], x[rows // 2, nq - 1, :], x[2, nq // 2, 0] = np.nan, np.inf, np.nan
    assert _run(kv_type, nq, nkv, hd, 16, seqs, x, K, V, False, entries) > 2


@pytest.mark.parametrize("kv_type", TYPES)
def test_prompt_nan_keys_that_a_part_sees_alone(kv_type):
    """Rows whose own position is the first of a wave's step or of a split tile's chunk."""
    x, K, V = _draw(5, [70], 2, 1, 64, kv_type, 70)
    K[0][32, 0, 3] = np.nan                                                 # row 32 and later
    assert _run(kv_type, 2, 1, 64, 16, [(70, 70)], x, K, V, False) == 2 * 38
    # 17 steps of 64 in three chunks: the third begins at position 768
    x, K, V = _draw(6, [1030], 2, 1, 64, kv_type, 262)
    K[0][768, 0, 3] = np.nan
    assert _run(kv_type, 2, 1, 64, 16, [(262, 1030)], x, K, V, False) == 2 * 262
    x, K, V = _draw(7, [1030], 2, 1, 64, kv_type, 300)
    K[0][768, 0, 3] = np.nan
    assert _run(kv_type, 2, 1, 64, 16, [(300, 1030)], x, K, V, False) == 2 * 262


@pytest.mark.parametrize("kv_type", TYPES)
@pytest.mark.parametrize("what", ["k", "v", "inf"])
@pytest.mark.parametrize("nq,nkv,hd,seqs", [
    (4, 1, 64, [(1, 6000)]), (4, 1, 64, [(9, 6000)]), (4, 1, 128, [(130, 6000)]),
    (64, 4, 64, [(40, 6000), (300, 300), (250, 250), (400, 420), (330, 330), (100, 100)])])
def test_parts_of_no_weight_bring_what_has_no_value(kv_type, what, nq, nkv, hd, seqs):
    """The first positions score 600 below the others, so that their part's weight underflows: a NaN key, or
    a value that is NaN or infinite, is seen all the same (0 x NaN and 0 x inf are NaN)."""
    rows = sum(a for a, _ in seqs)
    x, K, V = _draw(8, [n for _, n in seqs], nq, nkv, hd, kv_type, rows)
    x[:, :, 0] = 30.0
    for b in range(len(seqs)):
        K[b][:, :, 0] = 0.0
    K[0][:2000, :, 0] = -20.0
    if what == "k":
        K[0][100, 0, 5] = np.nan
    else:
        V[0][100, 0, 5] = np.nan if what == "v" else np.inf
    scale = 1.0

    def run(decode):
        c = Paged(kv_type, K, V, 16, nkv, hd, np.random.default_rng(58))
        start = np.concatenate([[0], np.cumsum([a for a, _ in seqs])]).astype(np.int32)
        xd = dev(x.reshape(rows, nq * hd))
        o = torch.full((rows, nq * hd), 77.0, device="cuda")
        ws = D.attn_workspace(q.OP_ATTN_PROMPT, len(seqs), nq, nkv, hd)
        if decode:
            q.qgemv_attn(*c.args(), c.kv_len, len(seqs), xd, nq * hd, nq, scale, o, ws)
        else:
            q.qgemv_attn_prompt(*c.args(), dev(start), c.kv_len, len(seqs), xd, nq * hd, rows, nq, scale, o, ws)
        return host(o).reshape(rows, nq, hd)

    for decode in ([True, False] if rows == 1 else [False]):
        say(f"no weight type={kv_type} {what} seqs={seqs[:3]} decode={decode}")
        got = run(decode)
        a, g = seqs[0][0], nq // nkv
        hit = got[:a, :g] if what == "k" else got[:a, :g, 5]
        assert not np.isfinite(hit).any()
        assert np.isfinite(got[a:]).all() and np.isfinite(got[:a, g:]).all()
        if what != "k":
            assert np.isfinite(np.delete(got[:a, :g], 5, axis=2)).all()
