"""The paged key-value cache and the attentions over it on the GPU, against their definitions in
64 bits (attn_common)."""
import numpy as np
import pytest

from gpu_common import dev, host, require_gpu, say, torch

import dequant_gemv_q4_amd as q
from dequant_gemv_q4_amd import device as D
from attn_common import Paged, TORCH, attention64, check_attention, rounded

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _draw(rng, lens, nkv, hd, kv_type, spread=1.0):
    K = [rounded(rng.standard_normal((n, nkv, hd)) * spread, kv_type) for n in lens]
    V = [rounded(rng.standard_normal((n, nkv, hd)), kv_type) for n in lens]
    return K, V


def _cat(parts):
    return tuple(np.stack([p[i].reshape(-1) for p in parts]) for i in range(3))


# ------------------------------------------------------------------------------------- one token

def _decode(kv_type, nq, nkv, hd, page, lens, seed, scale=None, qmul=1.0, **kw):
    say(f"attn type={kv_type} nq={nq} nkv={nkv} hd={hd} page={page} lens={lens[:8]}")
    rng = np.random.default_rng([77, seed])
    scale = hd ** -0.5 if scale is None else scale
    K, V = _draw(rng, lens, nkv, hd, kv_type)
    c = Paged(kv_type, K, V, page, nkv, hd, rng, **kw)
    n = len(lens)
    width = (nq + 2 * nkv) * hd
    qkv = (rng.standard_normal((n, width)) * qmul).astype(np.float32)
    o = torch.full((n, nq * hd), float("nan"), device="cuda")
    ws = D.attn_workspace(q.OP_ATTN, n, nq, nkv, hd)
    q.qgemv_attn(*c.args(), c.kv_len, n, dev(qkv), width, nq, scale, o, ws)
    ref, A, S = _cat([attention64(qkv[b, :nq * hd].reshape(nq, hd), K[b], V[b], nkv, scale,
                                  lens[b] - 1) for b in range(n)])
    check_attention(host(o), ref, A, S, lens, hd, kv_type, "attn")
    assert q.qgemv_attn_error(ws) == 0
    for b in range(n):
        if lens[b] == 0:
            assert not host(o)[b].any()


LENS = [1, 2, 15, 16, 17, 31, 32, 33, 0, 63, 64, 65, 127, 128, 130, 257]


@pytest.mark.parametrize("kv_type", [q.F16, q.BF16])
@pytest.mark.parametrize("nq,nkv,hd,page", [(12, 2, 128, 16), (8, 8, 64, 32), (5, 1, 96, 16),
                                            (20, 1, 64, 64), (40, 2, 128, 128), (4, 2, 256, 16),
                                            (6, 3, 192, 256)])
def test_attn_small_lengths(kv_type, nq, nkv, hd, page):
    _decode(kv_type, nq, nkv, hd, page, LENS, hd + page)


@pytest.mark.parametrize("kv_type,nq,nkv,hd,page,lens", [
    (q.F16, 12, 2, 128, 16, [5000]),
    (q.BF16, 12, 2, 128, 16, [4097, 1, 0, 700]),
    (q.BF16, 8, 4, 64, 64, [1500] * 9),
    (q.F16, 17, 1, 96, 32, [3001, 2]),
    (q.F16, 2, 2, 256, 128, [2049, 2047]),
    (q.BF16, 3, 1, 192, 256, [20001]),
])
def test_attn_long(kv_type, nq, nkv, hd, page, lens):
    _decode(kv_type, nq, nkv, hd, page, lens, len(lens))


def test_attn_many_sequences():
    rng = np.random.default_rng(3)
    _decode(q.BF16, 4, 2, 64, 16, [int(v) for v in rng.integers(0, 40, 1024)], 5)


def test_attn_sharp_scores_and_negative_scale():
    """Scores of a hundred units (one position takes all), a negative and a zero scale."""
    _decode(q.F16, 4, 2, 128, 16, [300, 77], 1, scale=1.0, qmul=4.0)
    _decode(q.BF16, 4, 2, 128, 16, [300, 77], 2, scale=-0.09)
    _decode(q.F16, 4, 2, 64, 16, [300, 77], 3, scale=0.0)
    _decode(q.F16, 4, 2, 64, 16, [300, 77], 4, scale=1e-6, qmul=1e6)
    _decode(q.F16, 4, 2, 64, 16, [300, 77], 5, scale=1e6, qmul=1e-6)


def test_attn_page_stride_and_table_rubbish():
    """A pool with gaps between the blocks; entries behind the last page hold any number."""
    _decode(q.F16, 12, 2, 128, 16, [100, 33, 16], 9, page_stride=2 * 128 * 16 * 3 + 8, bad_entry=2 ** 30)


def test_attn_offsets_beyond_32_bits():
    """Pages more than 2^32 elements into the pool."""
    hd, nkv, page, nq, n = 128, 1, 16, 4, 40
    stride = 3 << 30
    rng = np.random.default_rng(8)
    K, V = _draw(rng, [n], nkv, hd, q.F16)
    c = Paged(q.F16, K, V, page, nkv, hd, rng, spare=0)
    assert c.n_pages == 3
    pools = []
    for a in (c.k, c.v):
        big = torch.empty(2 * stride + page * hd, dtype=torch.float16, device="cuda")
        for p in range(3):
            big[p * stride:p * stride + page * hd] = a[p]
        pools.append(big)
    x = rng.standard_normal((1, nq * hd)).astype(np.float32)
    o = torch.empty((1, nq * hd), device="cuda")
    ws = D.attn_workspace(q.OP_ATTN, 1, nq, nkv, hd)
    q.qgemv_attn(q.F16, pools[0], pools[1], 3, page, stride, nkv, hd, c.table, c.max_pages, c.kv_len,
                 1, dev(x), nq * hd, nq, 0.1, o, ws)
    ref, A, S = _cat([attention64(x.reshape(nq, hd), K[0], V[0], nkv, 0.1, n - 1)])
    check_attention(host(o), ref, A, S, [n], hd, q.F16, "far pages")
    # and the append and the prompt form of the same token
    new = rng.standard_normal((1, 2 * hd)).astype(np.float32)
    nd = dev(new)
    one = torch.tensor([n], dtype=torch.int32, device="cuda")
    q.qgemv_kv_append(q.F16, pools[0], pools[1], 3, page, stride, nkv, hd, c.table, c.max_pages, None,
                      one, 1, nd, nd[:, hd:], 2 * hd, 1, ws)
    K[0][n - 1], V[0][n - 1] = rounded(new[:, :hd], q.F16), rounded(new[:, hd:], q.F16)
    ref, A, S = _cat([attention64(x.reshape(nq, hd), K[0], V[0], nkv, 0.1, n - 1)])
    wp = D.attn_workspace(q.OP_ATTN_PROMPT, 1, nq, nkv, hd)
    q.qgemv_attn_prompt(q.F16, pools[0], pools[1], 3, page, stride, nkv, hd, c.table, c.max_pages,
                        torch.tensor([0, 1], dtype=torch.int32, device="cuda"), one, 1, dev(x), nq * hd,
                        1, nq, 0.1, o, wp)
    check_attention(host(o), ref, A, S, [n], hd, q.F16, "far pages, prompt")


def test_attn_bad_pages_are_left_out():
    """An entry outside the pool, and a length beyond the table: those positions count as masked and
    the flag is set, once."""
    hd, nkv, nq, page = 64, 2, 4, 16
    rng = np.random.default_rng(4)
    K, V = _draw(rng, [100, 50, 64], nkv, hd, q.F16)
    c = Paged(q.F16, K, V, page, nkv, hd, rng, extra_entries=0, spare=0)
    c.table[0, 2] = c.n_pages               # positions 32..47 of sequence 0
    c.table[1, 0] = -7                      # positions 0..15 of sequence 1
    lens = [100, 50, 10 ** 6]               # sequence 2: its table ends at max_pages * page
    c.table[2, 4:] = -1
    x = rng.standard_normal((3, nq * hd)).astype(np.float32)
    keep = [np.r_[0:32, 48:100], np.r_[16:50], np.r_[0:64]]
    parts = [attention64(x[b].reshape(nq, hd), K[b][keep[b]], V[b][keep[b]], nkv, 0.125,
                         len(keep[b]) - 1) for b in range(3)]
    ref, A, S = _cat(parts)
    kv = torch.tensor(lens, dtype=torch.int32, device="cuda")
    for prompt in (False, True):
        say(f"bad pages prompt={prompt}")
        o = torch.full((3, nq * hd), float("nan"), device="cuda")
        ws = D.attn_workspace(q.OP_ATTN_PROMPT if prompt else q.OP_ATTN, 3, nq, nkv, hd)
        if prompt:
            q.qgemv_attn_prompt(*c.args(), torch.arange(4, dtype=torch.int32, device="cuda"), kv, 3,
                                dev(x), nq * hd, 3, nq, 0.125, o, ws)
        else:
            q.qgemv_attn(*c.args(), kv, 3, dev(x), nq * hd, nq, 0.125, o, ws)
        check_attention(host(o), ref, A, S, [100, 50, 64], hd, q.F16, "bad pages")
        assert q.qgemv_attn_error(ws) == 1
        assert q.qgemv_attn_error(ws) == 0


def test_attn_all_pages_bad_gives_zero():
    rng = np.random.default_rng(5)
    K, V = _draw(rng, [40, 40], 1, 64, q.BF16)
    c = Paged(q.BF16, K, V, 16, 1, 64, rng)
    c.table[0] = -1
    x = dev(rng.standard_normal((2, 128)).astype(np.float32))
    for op in (q.OP_ATTN, q.OP_ATTN_PROMPT):
        o = torch.full((2, 128), float("nan"), device="cuda")
        ws = D.attn_workspace(op, 2, 2, 1, 64)
        if op == q.OP_ATTN:
            q.qgemv_attn(*c.args(), c.kv_len, 2, x, 128, 2, 0.125, o, ws)
        else:
            q.qgemv_attn_prompt(*c.args(), torch.arange(3, dtype=torch.int32, device="cuda"), c.kv_len,
                                2, x, 128, 2, 2, 0.125, o, ws)
        assert not host(o)[0].any() and np.isfinite(host(o)[1]).all() and host(o)[1].any()
        assert q.qgemv_attn_error(ws) == 1


# --------------------------------------------------------------------------------------- prompts

def _prompt(kv_type, nq, nkv, hd, page, seqs, seed, tail=0, qmul=1.0, K=None, V=None, check=None):
    """seqs: (new rows, cached positions with them); tail rows behind the last sequence."""
    say(f"prompt type={kv_type} nq={nq} nkv={nkv} hd={hd} page={page} seqs={seqs[:6]}")
    rng = np.random.default_rng([78, seed])
    scale = hd ** -0.5
    lens = [b for _, b in seqs]
    if K is None:
        K, V = _draw(rng, [max(0, b) for b in lens], nkv, hd, kv_type)
    c = Paged(kv_type, K, V, page, nkv, hd, rng)
    start = np.concatenate([[0], np.cumsum([a for a, _ in seqs])]).astype(np.int32)
    rows = int(start[-1]) + tail
    width = (nq + 2 * nkv) * hd
    qkv = (rng.standard_normal((rows, width)) * qmul).astype(np.float32)
    o = torch.full((rows, nq * hd), 123.5, device="cuda")
    ws = D.attn_workspace(q.OP_ATTN_PROMPT, len(seqs), nq, nkv, hd)
    q.qgemv_attn_prompt(*c.args(), dev(start), dev(np.array(lens, np.int32)), len(seqs), dev(qkv),
                        width, rows, nq, scale, o, ws)
    got = host(o)
    assert (got[start[-1]:] == 123.5).all()
    parts, seen = [], []
    for b, (a, n) in enumerate(seqs):
        for i in range(a):
            last = n - a + i
            parts.append(attention64(qkv[start[b] + i, :nq * hd].reshape(nq, hd), K[b], V[b], nkv, scale,
                                     last))
            seen.append(max(0, last + 1))
    if not parts:
        return
    ref, A, S = _cat(parts)
    if check is not None:
        check(got[:start[-1]], ref, seen)
        return
    check_attention(got[:start[-1]], ref, A, S, seen, hd, kv_type, "prompt")
    for r, n in enumerate(seen):
        if n == 0:
            assert not got[r].any()
    assert q.qgemv_attn_error(ws) == 0


@pytest.mark.parametrize("kv_type", [q.F16, q.BF16])
@pytest.mark.parametrize("nq,nkv,hd,page", [(12, 2, 128, 16), (8, 8, 64, 32), (5, 1, 96, 16),
                                            (20, 1, 64, 64), (4, 2, 256, 16), (6, 3, 192, 256)])
def test_prompt_small(kv_type, nq, nkv, hd, page):
    _prompt(kv_type, nq, nkv, hd, page,
            [(1, 1), (2, 2), (0, 0), (7, 7), (31, 31), (33, 40), (1, 66), (5, 130), (0, 9), (64, 64)],
            hd + page, tail=3)


@pytest.mark.parametrize("kv_type,nq,nkv,hd,page,seqs", [
    (q.F16, 4, 2, 128, 16, [(300, 300), (1, 500), (129, 700)]),
    (q.BF16, 6, 1, 64, 64, [(257, 257)]),
    (q.F16, 3, 3, 96, 32, [(200, 333)]),
    (q.BF16, 2, 1, 256, 128, [(150, 1200)]),
    (q.F16, 8, 1, 128, 16, [(3, 9000)]),              # few rows over a long cache
    (q.BF16, 24, 2, 64, 16, [(17, 5000), (2, 3000)]),
])
def test_prompt_long(kv_type, nq, nkv, hd, page, seqs):
    _prompt(kv_type, nq, nkv, hd, page, seqs, len(seqs), tail=1)


def test_prompt_padded_rows_attend_to_nothing():
    """kv_len below the new rows (a padded batch): the first rows are at negative positions."""
    _prompt(q.F16, 4, 2, 64, 16, [(5, 2), (3, 0), (40, 39), (2, -3)], 1, tail=2)


def test_prompt_many_sequences():
    rng = np.random.default_rng(6)
    _prompt(q.BF16, 2, 1, 64, 16, [(int(a), int(a + c)) for a, c in zip(rng.integers(0, 4, 1024),
                                                                         rng.integers(0, 20, 1024))], 7)


def test_prompt_later_positions_do_not_reach_earlier_rows():
    """Infinities and NaN at a position reach the rows that see it and none before."""
    for hd, kv_type, bad in ((64, q.F16, np.inf), (128, q.BF16, np.nan), (128, q.F16, -np.inf)):
        rng = np.random.default_rng(11)
        n, at = 70, 41
        K, V = _draw(rng, [n], 1, hd, kv_type)
        V[0][at, 0, 5] = bad
        K[0][60, 0, 3] = np.nan

        def check(got, ref, seen, hd=hd, bad=bad):
            got = got.reshape(n, 2, hd)
            ref = ref.reshape(n, 2, hd)
            assert np.isfinite(got[:at]).all()
            assert np.abs(got[:at] - ref[:at]).max() < 1e-4
            mid = got[at:60]
            assert np.isfinite(np.delete(mid, 5, axis=2)).all()
            assert (np.isnan(mid[:, :, 5]) if np.isnan(bad) else mid[:, :, 5] == bad).all()
            assert np.isnan(got[60:]).all()

        with np.errstate(all="ignore"):
            _prompt(kv_type, 2, 1, hd, 16, [(n, n)], 3, K=K, V=V, check=check)


def test_bad_q_start_stays_in_bounds():
    """Row starts that fall or run past n_rows are cut to the rows there are."""
    rng = np.random.default_rng(12)
    K, V = _draw(rng, [30, 30, 30], 1, 64, q.F16)
    c = Paged(q.F16, K, V, 16, 1, 64, rng)
    x = dev(rng.standard_normal((8, 64)).astype(np.float32))
    ws = D.attn_workspace(q.OP_ATTN_PROMPT, 3, 1, 1, 64)
    for starts in ([0, 100, 3, 2 ** 31 - 1], [-5, 4, 2, 8], [7, 5, 3, 1], [-2 ** 31, -1, 0, 2 ** 31 - 1]):
        say(f"bad starts {starts}")
        guard = torch.full((24, 64), 7.0, device="cuda")
        o = guard[8:16]
        st = torch.tensor(starts, dtype=torch.int32, device="cuda")
        q.qgemv_attn_prompt(*c.args(), st, c.kv_len, 3, x, 64, 8, 1, 0.1, o, ws)
        q.qgemv_kv_append(*c.args(), st, c.kv_len, 3, x, x, 64, 8, ws)
        g = host(guard)
        assert (g[:8] == 7.0).all() and (g[16:] == 7.0).all()


# ---------------------------------------------------------------------------------------- append

def _append(kv_type, nkv, hd, page, seqs, decode, seed, special=False, nq=1, tail=0):
    say(f"append type={kv_type} nkv={nkv} hd={hd} page={page} seqs={seqs[:6]} decode={decode}")
    rng = np.random.default_rng([79, seed])
    lens = [b for _, b in seqs]
    zero = [np.full((max(0, n), nkv, hd), 3.25, np.float32) for n in lens]
    c = Paged(kv_type, zero, zero, page, nkv, hd, rng, fill=-2.5)
    start = np.concatenate([[0], np.cumsum([a for a, _ in seqs])]).astype(np.int32)
    rows = int(start[-1]) + tail
    width = (nq + 2 * nkv) * hd
    src = rng.standard_normal((rows, width)).astype(np.float32)
    if special:
        vals = np.array([np.inf, -np.inf, np.nan, 0.0, -0.0, 1e30, -1e30, 65519.9, 65520.0, 1 + 2.0 ** -11,
                         1 + 3 * 2.0 ** -11, 1 + 2.0 ** -8, 1 + 3 * 2.0 ** -9, 1e-7, 3e-8, 1e-39, 6e-5],
                        np.float32)
        src = rng.choice(vals, size=src.shape)
    kr = torch.from_numpy(src[:, nq * hd:(nq + nkv) * hd].copy()).to(TORCH[kv_type]).reshape(rows, nkv, hd)
    vr = torch.from_numpy(src[:, (nq + nkv) * hd:].copy()).to(TORCH[kv_type]).reshape(rows, nkv, hd)
    ek, ev = c.k.cpu().clone(), c.v.cpu().clone()
    ek4 = ek.reshape(c.n_pages, nkv, page, hd)
    ev4 = ev.reshape(c.n_pages, nkv, hd, page)
    for b, (a, n) in enumerate(seqs):
        for i in range(a):
            t = n - a + i
            if t >= 0:
                pg = c.table_host[b, t // page]
                ek4[pg, :, t % page] = kr[start[b] + i]
                ev4[pg, :, :, t % page] = vr[start[b] + i]
    sd = dev(src)
    ws = D.attn_workspace(q.OP_KV_APPEND, len(seqs), nq * nkv, nkv, hd)
    q.qgemv_kv_append(*c.args(), None if decode else dev(start), dev(np.array(lens, np.int32)),
                      len(seqs), sd[:, nq * hd:], sd[:, (nq + nkv) * hd:], width, rows, ws)
    torch.cuda.synchronize()
    for got, want in ((c.k.cpu(), ek), (c.v.cpu(), ev)):
        nan = torch.isnan(want)
        assert torch.equal(torch.isnan(got), nan)
        assert torch.equal(got.view(torch.int16)[~nan], want.view(torch.int16)[~nan])
    assert q.qgemv_attn_error(ws) == 0


@pytest.mark.parametrize("kv_type", [q.F16, q.BF16])
@pytest.mark.parametrize("nkv,hd,page", [(2, 128, 16), (8, 64, 32), (1, 96, 64), (3, 256, 16), (2, 192, 256)])
def test_append(kv_type, nkv, hd, page):
    _append(kv_type, nkv, hd, page, [(1, n) for n in (1, 2, 16, 17, 100, 33, 0)], True, hd)
    _append(kv_type, nkv, hd, page, [(1, 1), (0, 5), (7, 7), (8, 8), (9, 20), (40, 75), (3, 2), (0, 0), (65, 129)],
            False, page, nq=2, tail=4)


@pytest.mark.parametrize("kv_type", [q.F16, q.BF16])
def test_append_rounds_to_nearest_even(kv_type):
    _append(kv_type, 2, 64, 16, [(1, 3), (30, 41)], False, 1, special=True)


def test_append_many_sequences():
    rng = np.random.default_rng(9)
    a = rng.integers(0, 5, 1024)
    _append(q.BF16, 1, 64, 16, [(int(x), int(x + y)) for x, y in zip(a, rng.integers(0, 30, 1024))], False, 2)


def test_append_bad_pages_store_nothing():
    c = Paged(q.F16, [np.ones((40, 1, 64), np.float32)], [np.ones((40, 1, 64), np.float32)], 16, 1, 64,
              np.random.default_rng(0), extra_entries=0, fill=1.0)
    ws = D.attn_workspace(q.OP_KV_APPEND, 1, 1, 1, 64)
    x = torch.zeros((20, 128), device="cuda")
    start = torch.tensor([0, 20], dtype=torch.int32, device="cuda")
    good = int(c.table_host[0, 1])
    c.table[0, 2] = c.n_pages
    kv = torch.tensor([52], dtype=torch.int32, device="cuda")      # positions 32..51, 48.. behind the table
    q.qgemv_kv_append(*c.args(), start, kv, 1, x, x[:, 64:], 128, 20, ws)
    assert host((c.k == 1).all() & (c.v == 1).all())
    assert q.qgemv_attn_error(ws) == 1 and q.qgemv_attn_error(ws) == 0
    kv = torch.tensor([40], dtype=torch.int32, device="cuda")      # positions 20..39: 20..31 are stored
    q.qgemv_kv_append(*c.args(), start, kv, 1, x, x[:, 64:], 128, 20, ws)
    k = host(c.k.float()).reshape(c.n_pages, 16, 64)
    assert (k[good, 4:] == 0).all() and (k[good, :4] == 1).all()
    assert host(c.k == 0).sum() == 12 * 64 and host(c.v == 0).sum() == 12 * 64
    assert q.qgemv_attn_error(ws) == 1


def test_interleaved_pool():
    """K and V blocks side by side in one pool (page_stride of two blocks)."""
    nkv, hd, page, n = 2, 64, 16, 50
    block = nkv * hd * page
    rng = np.random.default_rng(13)
    pool = torch.full((4, 2 * block), float("nan"), dtype=torch.bfloat16, device="cuda")
    table = torch.tensor([[3, 0, 2, 1]], dtype=torch.int32, device="cuda")
    src = rng.standard_normal((n, 3 * nkv * hd)).astype(np.float32)
    sd = dev(src)
    start = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    kv = torch.tensor([n], dtype=torch.int32, device="cuda")
    ws = D.attn_workspace(q.OP_ATTN_PROMPT, 1, nkv, nkv, hd)
    cache = (q.BF16, pool, pool[:, block:], 4, page, 2 * block, nkv, hd, table, 4)
    q.qgemv_kv_append(*cache, start, kv, 1, sd[:, nkv * hd:], sd[:, 2 * nkv * hd:], 3 * nkv * hd, n, ws)
    o = torch.empty((n, nkv * hd), device="cuda")
    q.qgemv_attn_prompt(*cache, start, kv, 1, sd, 3 * nkv * hd, n, nkv, 0.125, o, ws)
    K = rounded(src[:, nkv * hd:2 * nkv * hd], q.BF16).reshape(n, nkv, hd)
    V = rounded(src[:, 2 * nkv * hd:], q.BF16).reshape(n, nkv, hd)
    ref, A, S = _cat([attention64(src[i, :nkv * hd].reshape(nkv, hd), K, V, nkv, 0.125, i) for i in range(n)])
    check_attention(host(o), ref, A, S, np.arange(1, n + 1), hd, q.BF16, "interleaved")
