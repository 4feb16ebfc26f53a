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


def test_attn_split_among_more_sequences_than_lanes():
    rng = np.random.default_rng(31)
    lens = [int(v) for v in rng.integers(0, 60, 150)]
    lens[3], lens[90], lens[149] = 9000, 1300, 700
    _decode(q.F16, 4, 1, 64, 16, lens, 6)


@pytest.mark.parametrize("kv_type,nq,nkv,hd,n_seq,long", [
    (q.F16, 8, 8, 64, 66, {0: 6000, 65: 1500}),       # over 64 sequences, 528 pairs for 512 slots
    (q.BF16, 8, 8, 64, 64, {40: 9000}),               # exactly as many pairs as slots
    (q.F16, 4, 4, 256, 64, {10: 3000, 11: 2999}),     # 256 slots
    (q.F16, 34, 2, 128, 129, {128: 5000, 3: 700}),    # two tiles of columns a KV head
])
def test_attn_more_pairs_than_slots_and_a_few_long(kv_type, nq, nkv, hd, n_seq, long):
    """Long sequences among so many others that nothing would be split for want of workgroups."""
    lens = [int(n) for n in np.random.default_rng(38).integers(1, 200, n_seq)]
    lens[7] = 0
    for b, n in long.items():
        lens[b] = n
    _decode(kv_type, nq, nkv, hd, 16, lens, n_seq)
    _decode(kv_type, nq, nkv, hd, 16, [300] * n_seq, n_seq + 1)


@pytest.mark.parametrize("kv_type,nq,nkv,hd,lens", [
    (q.F16, 40, 2, 128, [9000, 100, 3000]), (q.BF16, 66, 2, 64, [5000]), (q.F16, 17, 1, 256, [2500, 700, 0, 1]),
    (q.BF16, 40, 2, 96, [600 + i for i in range(130)] + [4000])])
def test_attn_tiles_side_by_side(kv_type, nq, nkv, hd, lens):
    """More than 16 query heads a KV head, with and without a split."""
    _decode(kv_type, nq, nkv, hd, 16, lens, 40)


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

def _prompt(kv_type, nq, nkv, hd, page, seqs, seed, tail=0, qmul=1.0, K=None, V=None, check=None,
            wide=False, scale=None):
    """seqs: (new rows, cached positions with them); tail rows behind the last sequence.  wide: sizes
    that the 128-row tiles take (many columns per sequence and a table of over 1024 positions)."""
    say(f"prompt type={kv_type} nq={nq} nkv={nkv} hd={hd} page={page} seqs={seqs[:6]} wide={wide}")
    if wide:
        assert sum(a for a, _ in seqs) * (nq // nkv) > 384 * len(seqs)
    rng = np.random.default_rng([78, seed])
    scale = hd ** -0.5 if scale is None else scale
    lens = [b for _, b in seqs]
    if K is None:
        K, V = _draw(rng, [max(0, b) for b in lens], nkv, hd, kv_type)
    c = Paged(kv_type, K, V, page, nkv, hd, rng, extra_entries=1024 // page + 1 if wide else 2)
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


@pytest.mark.parametrize("kv_type", [q.F16, q.BF16])
@pytest.mark.parametrize("nq,nkv,hd,page", [(12, 2, 128, 16), (10, 2, 64, 32), (5, 1, 96, 16),
                                            (20, 1, 64, 256), (4, 1, 256, 16), (6, 1, 192, 64)])
def test_prompt_wide(kv_type, nq, nkv, hd, page):
    """128-row tiles: a sequence ending inside a tile and a step, empty ones, single rows, a cached
    prefix, a padded one."""
    g = nq // nkv
    _prompt(kv_type, nq, nkv, hd, page,
            [(2100 // g, 2100 // g), (1, 1), (0, 0), (0, 9), (700 // g, 700 // g + 77), (3, 130), (30, 21)],
            hd + page, tail=3, wide=True)


@pytest.mark.parametrize("kv_type,nq,nkv,hd,page,seqs", [
    (q.F16, 8, 1, 128, 16, [(61, 5000)]),             # few tiles over a long cache: split over it
    (q.BF16, 24, 2, 64, 16, [(50, 4000), (50, 64)]),
    (q.F16, 4, 1, 256, 32, [(100, 2500)]),
    (q.BF16, 9, 1, 96, 16, [(45, 3333)]),
    (q.F16, 2, 1, 64, 16, [(1100, 1100)]),
])
def test_prompt_wide_long(kv_type, nq, nkv, hd, page, seqs):
    _prompt(kv_type, nq, nkv, hd, page, seqs, len(seqs), tail=1, wide=True)


def test_prompt_split_among_more_sequences_than_lanes():
    """16-column tiles of 100 sequences, 128-column tiles of 66, a few of them with long contexts."""
    rng = np.random.default_rng(32)
    seqs = [(int(a), int(a + c)) for a, c in zip(rng.integers(0, 3, 100), rng.integers(0, 30, 100))]
    seqs[70], seqs[99] = (2, 4000), (1, 2500)
    _prompt(q.BF16, 4, 1, 64, 16, seqs, 8, tail=1)
    seqs = [(25, 25 + int(c)) for c in rng.integers(0, 30, 66)]
    seqs[64], seqs[5] = (26, 3000), (0, 7)
    _prompt(q.F16, 16, 1, 64, 16, seqs, 9, wide=True)


def test_prompt_wide_more_tiles_than_are_resident():
    """128-column tiles in falling order of work: four sequences (tiles of 1 to 112 tiles' work), 70 of them
    (more than lanes), a padded and an empty one."""
    seqs = [(300, 300), (0, 40), (100, 900), (250, 250), (9, 4), (400, 420)]
    assert 4 * sum((a * 16 + 127) // 128 for a, _ in seqs) > 512
    _prompt(q.F16, 64, 4, 64, 32, seqs, 10, tail=2, wide=True)
    rng = np.random.default_rng(37)
    seqs = [(25 + int(c % 2), 25 + int(c)) for c in rng.integers(1, 60, 70)]
    seqs[66], seqs[3] = (60, 700), (0, 9)
    assert 2 * sum((a * 16 + 127) // 128 for a, _ in seqs) > 512
    _prompt(q.BF16, 32, 2, 64, 16, seqs, 11, tail=1, wide=True)


@pytest.mark.parametrize("kv_type,hd,seqs", [
    (q.F16, 64, [(40, 6000), (300, 300), (250, 250), (0, 5000), (400, 420), (9, 3000), (330, 330), (100, 100)]),
    (q.BF16, 128, [(10, 2600), (300, 300), (250, 250), (400, 420), (330, 330), (100, 100)]),
    (q.F16, 256, [(10, 2600), (300, 300), (250, 250), (12, 5)]),                    # 256 slots
    (q.BF16, 64, [(7, 3000)] + [(20, 25)] * 70 + [(9, 2500)]),                      # more than lanes
])
def test_prompt_wide_a_few_long_tiles_among_many(kv_type, hd, seqs):
    """More tiles than slots, of which those behind long contexts are split; their parts are joined within
    the launch."""
    nq, nkv = (96, 4) if len(seqs) > 64 else (64, 4)
    slots = 512 if hd <= 128 else 256
    assert nkv * (sum(a for a, _ in seqs) * (nq // nkv) // 128) >= slots
    _prompt(kv_type, nq, nkv, hd, 32, seqs, 14, tail=2, wide=True)


@pytest.mark.parametrize("n_seq", [70, 80])
def test_prompt_wide_tiles_that_fill_the_slots_only_when_counted(n_seq):
    """Sequences of four tiles, the last hardly begun: fewer pairs than slots by rows, more in fact, two behind
    long contexts."""
    rng = np.random.default_rng(39)
    seqs = [(25, 25 + int(c)) for c in rng.integers(0, 60, n_seq)]
    seqs[n_seq - 5], seqs[2] = (25, 5000), (25, 2500)
    assert 2 * (sum(a for a, _ in seqs) * 16 // 128) < 512 <= 2 * sum((a * 16 + 127) // 128 for a, _ in seqs)
    _prompt(q.BF16, 32, 2, 64, 16, seqs, 15, tail=1, wide=True)


def test_prompt_narrow_tiles_that_fill_the_slots():
    """16-column tiles, 512 for 512 slots, of which the longer sequence's are split."""
    _prompt(q.F16, 8, 8, 64, 16, [(500, 990), (497, 497)], 12)


def test_prompt_wide_many_heads_one_query_each():
    _prompt(q.F16, 3, 3, 128, 16, [(390, 400)], 2, wide=True)


@pytest.mark.parametrize("wide", [False, True])
def test_prompt_sharp_scores_and_other_scales(wide):
    """As for single tokens: scores of a hundred units, negative, zero, tiny and huge scales."""
    seqs = [(110, 300), (100, 131)] if wide else [(31, 300), (5, 77)]
    _prompt(q.F16, 4, 1, 128, 16, seqs, 1, wide=wide, scale=1.0, qmul=2.0)
    _prompt(q.BF16, 4, 1, 128, 16, seqs, 2, wide=wide, scale=-0.09)
    _prompt(q.F16, 4, 1, 64, 16, seqs, 3, wide=wide, scale=0.0)
    _prompt(q.BF16, 4, 1, 64, 16, seqs, 4, wide=wide, scale=-0.0)
    _prompt(q.F16, 4, 1, 64, 16, seqs, 5, wide=wide, scale=-1e-6, qmul=1e6)
    _prompt(q.F16, 4, 1, 64, 16, seqs, 6, wide=wide, scale=1e6, qmul=1e-6)
    _prompt(q.BF16, 4, 1, 64, 16, seqs, 7, wide=wide, scale=1e-40, qmul=1e-3)


@pytest.mark.parametrize("kv_type", [q.F16, q.BF16])
@pytest.mark.parametrize("top", [1e7, 2e7, 4e7, 8e7, 1.6e8, 3.2e8, 1e9, 1e12])
def test_scores_wider_apart_than_their_spread_stay_finite(kv_type, top):
    """Scores of 1e7 to 1e12 that grow slowly with the position: f32 spaces them by 1 to 2^17, and no
    rounding against the running maximum may leave the range of a weight.  The outputs have to be means of
    the values seen (sums of 400 terms and weights: 2^-14 covers 802 roundings); nearer than the scores'
    own rounding allows, the definition does not say which."""
    hd, nq, page, n, rows = 64, 4, 16, 400, 130
    rng = np.random.default_rng(36)
    for every in (24, 40):
        K = np.zeros((n, 1, hd), np.float32)
        K[:, 0, 0], K[:, 0, 1] = 1.0, np.arange(n) // every
        V = rounded(rng.standard_normal((n, 1, hd)), kv_type)
        x = np.zeros((rows, nq * hd), np.float32)
        x[:, 0::hd], x[:, 1::hd] = np.float32(top) * rng.uniform(0.9, 1.1, (rows, nq)), 1.0
        c = Paged(kv_type, [K], [V], page, 1, hd, rng, extra_entries=70)
        for count in (0, 12, rows):                  # single token, 16-column tiles, 128-row tiles
            say(f"large scores top={top} every={every} rows={count}")
            m = max(count, 1)
            xd, o = dev(x[:m]), torch.full((m, nq * hd), float("nan"), device="cuda")
            if count:
                ws = D.attn_workspace(q.OP_ATTN_PROMPT, 1, nq, 1, hd)
                q.qgemv_attn_prompt(*c.args(), torch.tensor([0, m], dtype=torch.int32, device="cuda"), c.kv_len, 1,
                                    xd, nq * hd, m, nq, 1.0, o, ws)
            else:
                ws = D.attn_workspace(q.OP_ATTN, 1, nq, 1, hd)
                q.qgemv_attn(*c.args(), c.kv_len, 1, xd, nq * hd, nq, 1.0, o, ws)
            last = [n - m + r for r in range(m)]
            got = host(o).reshape(m, nq, hd)
            assert np.isfinite(got).all()
            for r in range(m):
                seen = V[:last[r] + 1, 0]
                slack = 2.0 ** -14 * np.abs(seen).max(axis=0)
                assert (got[r] <= seen.max(axis=0) + slack).all() and (got[r] >= seen.min(axis=0) - slack).all()


def test_prompt_padded_rows_attend_to_nothing():
    """kv_len below the new rows (a padded batch): the first rows are at negative positions."""
    _prompt(q.F16, 4, 2, 64, 16, [(5, 2), (3, 0), (40, 39), (2, -3)], 1, tail=2)


@pytest.mark.parametrize("seqs", [
    [(200, 3000), (150, 0), (130, -3), (140, 139)],                         # split, joined by a second launch
    [(20, 4000), (400, 0), (300, 1200), (380, -1), (10, 0)],                # a few split among many
    [(400, 0), (300, 0), (400, 20)]])                                       # none
def test_prompt_wide_padded_rows_are_zero(seqs):
    """128-row tiles of sequences without positions: their rows are written, with zeros."""
    _prompt(q.F16, 64 if len(seqs) > 4 else 32, 8, 64, 16, seqs, 16, tail=2, wide=True)


def test_prompt_many_sequences():
    rng = np.random.default_rng(6)
    _prompt(q.BF16, 2, 1, 64, 16, [(int(a), int(a + c)) for a, c in zip(rng.integers(0, 4, 1024),
                                                                         rng.integers(0, 20, 1024))], 7)


def test_prompt_later_positions_do_not_reach_earlier_rows():
    """Infinities and NaN at a position make the rows that see it non-finite and no row before it."""
    for hd, kv_type, bad, n, at, kn in ((64, q.F16, np.inf, 70, 41, 60), (128, q.BF16, np.nan, 70, 41, 60),
                                        (128, q.F16, -np.inf, 70, 41, 60), (256, q.F16, np.inf, 70, 41, 60),
                                        (64, q.BF16, np.inf, 210, 100, 131), (96, q.F16, -np.inf, 210, 64, 65),
                                        (128, q.F16, np.nan, 210, 127, 190), (128, q.BF16, -np.inf, 210, 3, 205),
                                        (192, q.BF16, np.inf, 210, 150, 151), (256, q.BF16, np.nan, 210, 90, 120)):
        rng = np.random.default_rng(11)
        K, V = _draw(rng, [n], 1, hd, kv_type)
        V[0][at, 0, 5] = bad
        K[0][kn, 0, 3] = np.nan

        def check(got, ref, seen):
            got = got.reshape(n, 2, hd)
            ref = ref.reshape(n, 2, hd)
            assert np.isfinite(got[:at]).all()
            assert np.abs(got[:at] - ref[:at]).max() < 1e-4
            mid = got[at:kn]
            assert np.isfinite(np.delete(mid, 5, axis=2)).all()
            # an infinity may come out as NaN: a probability enters the product as p1 + p2, and with
            # p2 = 0 or of the other sign p1 inf + p2 inf is NaN
            assert (~np.isfinite(mid[:, :, 5])).all()
            assert np.isnan(got[kn:]).all()

        with np.errstate(all="ignore"):
            _prompt(kv_type, 2, 1, hd, 16, [(n, n)], 3, K=K, V=V, check=check, wide=n > 200)


def test_prompt_wide_bad_pages_are_left_out():
    hd, nq, page, n = 64, 4, 16, 150
    rng = np.random.default_rng(14)
    K, V = _draw(rng, [n], 1, hd, q.BF16)
    c = Paged(q.BF16, K, V, page, 1, hd, rng, extra_entries=70)
    c.table[0, 2] = c.n_pages                # positions 32..47
    c.table[0, 7] = -1                       # positions 112..127
    x = rng.standard_normal((n, nq * hd)).astype(np.float32)
    o = torch.full((n, nq * hd), float("nan"), device="cuda")
    ws = D.attn_workspace(q.OP_ATTN_PROMPT, 1, nq, 1, hd)
    q.qgemv_attn_prompt(*c.args(), torch.tensor([0, n], dtype=torch.int32, device="cuda"), c.kv_len, 1, dev(x),
                        nq * hd, n, nq, 0.125, o, ws)
    keep = np.r_[0:32, 48:112, 128:n]
    parts = [attention64(x[r].reshape(nq, hd), K[0][keep[keep <= r]], V[0][keep[keep <= r]], 1, 0.125,
                         int((keep <= r).sum()) - 1) for r in range(n)]
    ref, A, S = _cat(parts)
    check_attention(host(o), ref, A, S, np.arange(1, n + 1), hd, q.BF16, "bad pages, wide")
    assert q.qgemv_attn_error(ws) == 1 and q.qgemv_attn_error(ws) == 0


@pytest.mark.parametrize("kv_type,beyond", [(q.F16, 8), (q.F16, 300), (q.BF16, 300), (q.BF16, 2 ** 31 - 1 - 1040)])
def test_prompt_wide_table_ends_inside_a_step(kv_type, beyond):
    """Lengths beyond a table of 1040 positions (a step is 64): rows up to and behind its end see what
    the table has, and the flag is set."""
    hd, nq, page, n, cap = 64, 4, 16, 130, 1040
    rng = np.random.default_rng(35)
    K, V = _draw(rng, [cap], 1, hd, kv_type)
    c = Paged(kv_type, K, V, page, 1, hd, rng, extra_entries=0)
    assert c.max_pages * page == cap and n * nq > 384
    x = rng.standard_normal((n, nq * hd)).astype(np.float32)
    o = torch.full((n, nq * hd), float("nan"), device="cuda")
    ws = D.attn_workspace(q.OP_ATTN_PROMPT, 1, nq, 1, hd)
    q.qgemv_attn_prompt(*c.args(), torch.tensor([0, n], dtype=torch.int32, device="cuda"),
                        torch.tensor([cap + beyond], dtype=torch.int32, device="cuda"), 1, dev(x), nq * hd, n, nq,
                        0.125, o, ws)
    last = [min(cap + beyond - n + r, cap - 1) for r in range(n)]
    ref, A, S = _cat([attention64(x[r].reshape(nq, hd), K[0], V[0], 1, 0.125, last[r]) for r in range(n)])
    check_attention(host(o), ref, A, S, np.array(last) + 1, hd, kv_type, "table ends inside a step")
    assert q.qgemv_attn_error(ws) == 1 and q.qgemv_attn_error(ws) == 0


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


# ---------------------------------------------------------------- streams, graphs, shared workspaces

def _step(rng, kv_type, nq, nkv, hd, page, seqs, wide=False):
    """A call's tensors: a cache of the sequences and the packed QKV rows."""
    lens = [b for _, b in seqs]
    K, V = _draw(rng, lens, nkv, hd, kv_type)
    c = Paged(kv_type, K, V, page, nkv, hd, rng, fill=0.0, extra_entries=1024 // page + 1 if wide else 4)
    start = np.concatenate([[0], np.cumsum([a for a, _ in seqs])]).astype(np.int32)
    width = (nq + 2 * nkv) * hd
    qkv = dev(rng.standard_normal((int(start[-1]), width)).astype(np.float32))
    return c, dev(start), qkv, width, int(start[-1])


def test_one_workspace_serves_every_operation_in_turn():
    """Append, prompt (16-column and 128-row tiles, split and not) and single tokens share the largest
    workspace, again and again; every result is bit for bit that of a workspace of its own."""
    rng = np.random.default_rng(21)
    nq, nkv, hd = 8, 2, 128
    calls = []
    for seqs, wide in (([(1, 3000), (1, 40)], False), ([(5, 2000)], False), ([(120, 4000)], True), ([(1, 700)] * 5, False)):
        c, start, qkv, width, rows = _step(rng, q.F16, nq, nkv, hd, 16, seqs, wide)
        calls.append((c, start, qkv, width, rows, len(seqs), all(a == 1 for a, _ in seqs)))

    def run(call, ws):
        c, start, qkv, width, rows, n, decode = call
        o = torch.full((rows, nq * hd), float("nan"), device="cuda")
        q.qgemv_kv_append(*c.args(), None if decode else start, c.kv_len, n, qkv[:, nq * hd:],
                          qkv[:, (nq + nkv) * hd:], width, rows, ws)
        if decode:
            q.qgemv_attn(*c.args(), c.kv_len, n, qkv, width, nq, 0.09, o, ws)
        else:
            q.qgemv_attn_prompt(*c.args(), start, c.kv_len, n, qkv, width, rows, nq, 0.09, o, ws)
        return o

    alone = [host(run(call, D.attn_workspace(q.OP_ATTN_PROMPT, 8, nq, nkv, hd))) for call in calls]
    ws = D.attn_workspace(q.OP_ATTN_PROMPT, 8, nq, nkv, hd)
    for rep in range(4):
        outs = [run(call, ws) for call in calls]
        for o, ref in zip(outs, alone):
            assert np.array_equal(host(o), ref), rep


@pytest.mark.parametrize("seqs,wide", [([(1, 9000), (1, 17), (1, 2500)], False), ([(3, 6000), (2, 900)], False),
                                       ([(70, 6000)], True), ([(420, 420)], True),
                                       ([(200, 6000)] + [(600, 600)] * 9, True),
                                       ([(1, 20000)] + [(1, 30)] * 300, False)])
def test_repeated_calls_are_bitwise_identical(seqs, wide):
    rng = np.random.default_rng(22)
    nq, nkv, hd = 12, 2, 128
    c, start, qkv, width, rows = _step(rng, q.BF16, nq, nkv, hd, 16, seqs, wide)
    ws = D.attn_workspace(q.OP_ATTN_PROMPT, len(seqs), nq, nkv, hd)
    outs = []
    for _ in range(20):
        o = torch.full((rows, nq * hd), float("nan"), device="cuda")
        if all(a == 1 for a, _ in seqs):
            q.qgemv_attn(*c.args(), c.kv_len, len(seqs), qkv, width, nq, 0.09, o, ws)
        else:
            q.qgemv_attn_prompt(*c.args(), start, c.kv_len, len(seqs), qkv, width, rows, nq, 0.09, o, ws)
        outs.append(o)
    ref = host(outs[0])
    assert np.isfinite(ref).all()
    for o in outs[1:]:
        assert np.array_equal(host(o), ref)


def test_two_streams_with_workspaces_of_their_own():
    rng = np.random.default_rng(23)
    nq, nkv, hd = 8, 2, 64
    jobs = []
    for seqs in ([(1, 5000), (1, 300)], [(1, 900)] * 6):
        c, _, qkv, width, rows = _step(rng, q.F16, nq, nkv, hd, 16, seqs)
        jobs.append((c, qkv, width, rows, D.attn_workspace(q.OP_ATTN, len(seqs), nq, nkv, hd)))

    def run(job, stream=None):
        c, qkv, width, rows, ws = job
        o = torch.empty((rows, nq * hd), device="cuda")
        q.qgemv_attn(*c.args(), c.kv_len, rows, qkv, width, nq, 0.125, o, ws, stream=stream)
        return o

    refs = [host(run(j)) for j in jobs]
    streams = [torch.cuda.Stream() for _ in jobs]
    torch.cuda.synchronize()
    for _ in range(10):
        outs = [run(j, st) for j, st in zip(jobs, streams)]
        torch.cuda.synchronize()
        for o, ref in zip(outs, refs):
            assert np.array_equal(host(o), ref)


def test_graph_replays_follow_the_lengths_on_the_device():
    """A decode step (append, attention) and a prompt captured once; each replay has other lengths
    and rows, and eager work in between, and gives the eager call's bits."""
    rng = np.random.default_rng(24)
    nq, nkv, hd, n = 8, 2, 128, 4
    c, start, qkv, width, rows = _step(rng, q.F16, nq, nkv, hd, 16, [(1, 4000), (1, 100), (1, 900), (1, 33)])
    cp, pstart, pqkv, pwidth, prows = _step(rng, q.F16, nq, nkv, hd, 16, [(90, 400), (60, 200)])
    ws = D.attn_workspace(q.OP_ATTN_PROMPT, n, nq, nkv, hd)
    o = torch.empty((rows, nq * hd), device="cuda")
    po = torch.empty((prows, nq * hd), device="cuda")

    def run():
        q.qgemv_kv_append(*c.args(), None, c.kv_len, n, qkv[:, nq * hd:], qkv[:, (nq + nkv) * hd:], width, n, ws)
        q.qgemv_attn(*c.args(), c.kv_len, n, qkv, width, nq, 0.09, o, ws)
        q.qgemv_attn_prompt(*cp.args(), pstart, cp.kv_len, 2, pqkv, pwidth, prows, nq, 0.09, po, ws)

    run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run()
    for rep, (lens, plens, cut) in enumerate((((4000, 100, 900, 33), (400, 200), 90), ((0, 64, 1, 33), (90, 60), 10),
                                              ((3999, 0, 850, 20), (300, 150), 140))):
        c.kv_len.copy_(torch.tensor(lens, dtype=torch.int32))
        cp.kv_len.copy_(torch.tensor(plens, dtype=torch.int32))
        pstart.copy_(torch.tensor([0, cut, 150], dtype=torch.int32))
        qkv.normal_()
        k0, v0 = c.k.clone(), c.v.clone()
        o.fill_(-1)
        po.fill_(-1)
        g.replay()
        torch.cuda.synchronize()
        got = [host(t).copy() for t in (o, po, c.k.view(torch.int16), c.v.view(torch.int16))]
        c.k.copy_(k0)
        c.v.copy_(v0)
        o.fill_(-2)
        po.fill_(-2)
        run()
        torch.cuda.synchronize()
        for a, b in zip(got, (o, po, c.k.view(torch.int16), c.v.view(torch.int16))):
            assert np.array_equal(a, host(b)), rep


def test_graph_replays_where_the_batch_fills_the_slots():
    """70 sequences of one token and a prompt batch of more tiles than slots, captured once on one workspace:
    none split, a few split and only one left by turns, each with the eager call's bits."""
    rng = np.random.default_rng(41)
    nq, nkv, hd, n = 64, 8, 64, 70
    c, _, qkv, width, _ = _step(rng, q.BF16, nq, nkv, hd, 16, [(1, 3000)] + [(1, 300)] * (n - 2) + [(1, 1500)])
    pseqs = [(20, 4000), (400, 400), (300, 1200), (380, 380)]
    cp, pstart, pqkv, pwidth, prows = _step(rng, q.F16, nq, nkv, hd, 16, pseqs, True)
    assert nkv * (prows * (nq // nkv) // 128) >= 512
    ws = D.attn_workspace(q.OP_ATTN_PROMPT, n, nq, nkv, hd)
    o, po = torch.empty((n, nq * hd), device="cuda"), torch.empty((prows, nq * hd), device="cuda")

    def run():
        q.qgemv_attn(*c.args(), c.kv_len, n, qkv, width, nq, 0.09, o, ws)
        q.qgemv_attn_prompt(*cp.args(), pstart, cp.kv_len, len(pseqs), pqkv, pwidth, prows, nq, 0.09, po, ws)

    run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run()
    full = [3000] + [300] * (n - 2) + [1500]
    for rep, (lens, plens) in enumerate(((full, [4000, 400, 1200, 380]), ([200] * n, [20, 400, 300, 380]),
                                         ([3000] + [0] * (n - 1), [4000, 0, 0, 0]), (full, [3999, 400, 1200, 300]))):
        c.kv_len.copy_(torch.tensor(lens, dtype=torch.int32))
        cp.kv_len.copy_(torch.tensor(plens, dtype=torch.int32))
        qkv.normal_()
        o.fill_(-1)
        po.fill_(-1)
        g.replay()
        torch.cuda.synchronize()
        got = [host(t).copy() for t in (o, po)]
        o.fill_(-2)
        po.fill_(-2)
        run()
        torch.cuda.synchronize()
        for a, b in zip(got, (o, po)):
            assert np.isfinite(a).all() and np.array_equal(a, host(b)), rep
    assert q.qgemv_attn_error(ws) == 0


def test_two_graphs_share_a_workspace():
    rng = np.random.default_rng(25)
    nq, nkv, hd = 4, 1, 64
    ws = D.attn_workspace(q.OP_ATTN, 2, nq, nkv, hd)
    jobs = []
    for seqs in ([(1, 6000), (1, 3)], [(1, 2000)]):
        c, _, qkv, width, rows = _step(rng, q.BF16, nq, nkv, hd, 32, seqs)
        o = torch.empty((rows, nq * hd), device="cuda")
        run = (lambda c=c, qkv=qkv, width=width, rows=rows, o=o:
               q.qgemv_attn(*c.args(), c.kv_len, rows, qkv, width, nq, 0.125, o, ws))
        run()
        torch.cuda.synchronize()
        ref = host(o).copy()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run()
        jobs.append((g, o, ref, run))
    for rep in range(6):
        for g, o, ref, run in jobs:
            o.zero_()
            g.replay()
        torch.cuda.synchronize()
        for g, o, ref, run in jobs:
            assert np.array_equal(host(o), ref), rep
        jobs[rep % 2][3]()


def test_tensors_of_the_wrong_type_device_or_layout_are_refused():
    rng = np.random.default_rng(26)
    c, start, qkv, width, rows = _step(rng, q.F16, 4, 2, 64, 16, [(1, 30), (1, 7)])
    ws = D.attn_workspace(q.OP_ATTN, 2, 4, 2, 64)
    o = torch.empty((rows, 256), device="cuda")

    def call(**kw):
        a = dict(zip(("kv_type", "k", "v", "n_pages", "page", "stride", "nkv", "hd", "table", "max_pages"), c.args()))
        a.update(kv_len=c.kv_len, n_seq=2, q=qkv, q_stride=width, nq=4, scale=0.1, o=o, ws=ws)
        a.update(kw)
        q.qgemv_attn(*a.values())

    call()
    wide = torch.zeros((2, c.max_pages + 3), dtype=torch.int32, device="cuda")
    for kw in (dict(kv_len=c.kv_len.long()), dict(table=c.table.long()), dict(table=wide[:, :c.max_pages]),
               dict(kv_len=c.kv_len.cpu()), dict(q=qkv.half()), dict(o=o.cpu()), dict(k=c.k.bfloat16()),
               dict(kv_type=q.BF16), dict(ws=ws.cpu()), dict(o=torch.empty((rows, 512), device="cuda")[:, ::2])):
        with pytest.raises(TypeError):
            call(**kw)
    z = torch.zeros((4, 8), device="cuda")
    ids, w = torch.zeros((4, 2), dtype=torch.int32, device="cuda"), torch.zeros((4, 2), device="cuda")
    q.qgemv_route(z, 4, 8, 0, None, 1, 1, 1, 2, True, 1.0, ids, w)
    for args in ((z.double(), ids, w), (z, ids.long(), w), (z, ids, w.half()), (z.cpu(), ids, w)):
        with pytest.raises(TypeError):
            q.qgemv_route(args[0], 4, 8, 0, None, 1, 1, 1, 2, True, 1.0, args[1], args[2])
    with pytest.raises(q.QgemvError):
        q.qgemv_route(z, 4, 8, 0, None, 1, 1, 1, 9, True, 1.0, ids, w)
    with pytest.raises(q.QgemvError):
        call(ws=None)
