"""Attention of a batch whose sequences begin alike, on the GPU, against the definition in 64 bits with each
sequence's positions spelled out (kv_common)."""
import ctypes

import numpy as np
import pytest

from gpu_common import dev, host, require_gpu, say, torch

import dequant_gemv_q4_amd as q
from dequant_gemv_q4_amd import device as D
from kv_common import ALL, BYTES, Cache, check_rows, held, parts64, scales64
from test_gpu_kv8 import _draw, ints

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def shared(kv_type, nq, nkv, hd, page, groups, seed=0, outside=(0, 0), scale=None, extra_entries=2, lens=None,
           bad_rest=False, gap=0, spread=1.0):
    """groups: lists of (shared positions, cached positions of its own behind them) of each sequence, the
    largest share first.  outside: sequences before the first and behind the last group."""
    say(f"shared type={kv_type} nq={nq} nkv={nkv} hd={hd} page={page} groups={[g[:3] for g in groups[:4]]}")
    rng = np.random.default_rng([93, seed])
    scale = hd ** -0.5 if scale is None else scale
    K, V, tables, starts, share = [], [], {}, [outside[0]], []
    for i in range(outside[0]):
        k, v = _draw(rng, [17 + 30 * i], nkv, hd, spread)
        K += k
        V += v
        share.append(9)                                     # not of a group: it shares nothing
    for g in groups:
        first = len(K)
        for i, (s, own) in enumerate(g):
            k, v = _draw(rng, [s + own], nkv, hd, spread)
            if i:
                k[0][:s], v[0][:s] = K[first][:s], V[first][:s]
                for e in range(s // page):
                    tables[(first + i, e)] = (first, e)
            K += k
            V += v
            share.append(s)
        starts.append(len(K))
    for i in range(outside[1]):
        k, v = _draw(rng, [40 + i], nkv, hd, spread)
        K += k
        V += v
        share.append(33)
    c = Cache(kv_type, K, V, page, nkv, hd, rng, extra_entries=extra_entries, tables=tables, gap=gap)
    if bad_rest:                                            # the others' entries of the prefix are not read
        for (b, e) in tables:
            c.table[b, e] = -5
    n = len(K)
    kv = c.kv_len if lens is None else ints(lens)
    length = [len(k) for k in K] if lens is None else lens
    width = (nq + 2 * nkv) * hd
    x = rng.standard_normal((n, width)).astype(np.float32)
    o = torch.full((n, nq * hd), float("nan"), device="cuda")
    ws = D.attn_workspace(q.OP_ATTN_SHARED, n, nq, nkv, hd)
    q.qgemv_attn_shared(*c.args(), kv, n, ints(starts), ints(share), len(groups), dev(x), width, nq, scale, o, ws)
    parts = []
    for b in range(n):
        hk, hv = held(K[b], kv_type), held(V[b], kv_type)
        dv = scales64(V[b], kv_type) if kv_type in BYTES and len(V[b]) else np.ones(V[b].shape[:2])
        qr = x[b, :nq * hd].reshape(nq, hd)
        parts.append(parts64(qr, hk, hv, dv, nkv, scale, length[b] - 1, kv_type))
    check_rows(host(o), parts, length, hd, kv_type, "shared")
    assert q.qgemv_attn_error(ws) == 0
    return c, x, host(o)


@pytest.mark.parametrize("kv_type", ALL)
@pytest.mark.parametrize("nq,nkv,hd,page", [(12, 2, 128, 16), (8, 8, 64, 32), (5, 1, 96, 16), (20, 1, 64, 64),
                                            (40, 2, 128, 128), (4, 2, 256, 16), (6, 3, 192, 256)])
def test_shared_small(kv_type, nq, nkv, hd, page):
    """Prefixes that end at, before and behind page and tile borders, groups of one, none shared, no tail."""
    groups = [[(64, 5), (64, 1), (64, 200)], [(33, 7)], [(0, 9), (0, 0), (0, 70)], [(130, 0), (130, 3), (100, 31)],
              [(16, 1), (15, 1), (1, 1), (0, 2)], [(257, 90), (257, 300), (256, 1), (255, 64)]]
    shared(kv_type, nq, nkv, hd, page, groups, hd + page, outside=(2, 1))


@pytest.mark.parametrize("kv_type,nq,nkv,hd,page,groups", [
    (q.F16, 12, 2, 128, 16, [[(3000, 40)] * 9]),
    (q.BF16, 8, 4, 64, 64, [[(1500, 700), (1500, 3)] * 4, [(2000, 20)] * 5]),
    (q.I8, 16, 1, 128, 32, [[(5000, 100)] * 20]),
    (q.F8, 24, 8, 64, 16, [[(1800, 100), (1700, 130)] * 16]),
    (q.F16, 40, 2, 96, 32, [[(900, 9)] * 3, [(4000, 1)] * 2]),
    (q.F8, 4, 1, 256, 64, [[(2500, 60)] * 40]),
    (q.BF16, 14, 2, 192, 16, [[(777, 33)] * 11, [(778, 2000), (778, 1)]]),
    (q.I8, 2, 1, 64, 16, [[(9000, 1)] * 2]),
])
def test_shared_long(kv_type, nq, nkv, hd, page, groups):
    shared(kv_type, nq, nkv, hd, page, groups, len(groups))


def form_of(kv_type, n_seq, n_group, nq, nkv, hd, positions):
    """Which kernels take the call (the launcher's own choice): 16-column tiles, 128-column tiles with parts, split
    few among many, or whole."""
    fn = ctypes.CDLL(q.LIB_PATH)["_ZN2qg11shared_formEiliiiil"]
    fn.restype = ctypes.c_int
    fn.argtypes = [ctypes.c_int, ctypes.c_int64, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int64]
    return ["16", "parted", "few", "whole"][fn(kv_type, n_seq, n_group, nq, nkv, hd, positions)]


@pytest.mark.parametrize("kv_type", ALL)
@pytest.mark.parametrize("form,nq,nkv,hd,page,groups,outside", [
    ("parted", 64, 2, 128, 16, [[(1003, 3 + i % 9) for i in range(60)], [(77, 40), (70, 3)] * 36], (1, 2)),
    ("parted", 128, 1, 64, 32, [[(1200, 1 + 7 * i % 40) for i in range(66)]], (0, 0)),
    ("parted", 60, 3, 96, 16, [[(150, 2)] * 90 + [(17, 900)], [(5, 1)] * 50], (3, 0)),
    ("parted", 64, 1, 192, 64, [[(130, 9)] * 100, [(700, 3), (0, 7), (700, 2)] * 10], (0, 1)),
    ("parted", 64, 2, 256, 64, [[(1030, 9)] * 20, [(64, 1), (64, 70)] * 56], (0, 0)),
    ("few", 64, 16, 64, 16, [[(20 + 4 * i, i % 5), (20 + 4 * i, 2), (9, 1)] for i in range(43)] + [[(1900, 5)] * 3],
     (1, 1)),
    ("few", 64, 8, 256, 32, [[(40, 4)] * 2 for _ in range(66)] + [[(1100, 20), (1100, 1)]], (0, 0)),
    ("whole", 64, 16, 64, 16, [[(9 + 3 * i, i % 7)] * 3 for i in range(45)], (2, 0)),
])
def test_shared_by_128_columns(kv_type, form, nq, nkv, hd, page, groups, outside):
    """Groups of more rows than 16-column tiles take, and more groups than workgroup slots."""
    n = sum(len(g) for g in groups) + sum(outside)
    lens = [s + a for g in groups for s, a in g] + [17 + 30 * i for i in range(outside[0])] + [41] * outside[1]
    positions = (-(-max(lens) // page) + 2) * page
    assert form_of(kv_type, n, len(groups), nq, nkv, hd, positions) == form
    shared(kv_type, nq, nkv, hd, page, groups, 11, outside=outside)


@pytest.mark.parametrize("kv_type,nq,nkv,hd,n,prefix", [
    (q.F16, 32, 8, 64, 60, 4500), (q.BF16, 16, 1, 128, 40, 7000), (q.I8, 32, 2, 128, 100, 10000)])
def test_shared_much_work(kv_type, nq, nkv, hd, n, prefix):
    """Enough work for the 128-column tiles in a few rows."""
    groups = [[(prefix, 1 + i % 50) for i in range(n)]]
    positions = (-(-(prefix + 50) // 32) + 2) * 32
    assert form_of(kv_type, n, 1, nq, nkv, hd, positions) == "parted"
    shared(kv_type, nq, nkv, hd, 32, groups, 14)


def test_choice_of_form():
    """By the work, the type and the groups; what the sums of halves meet on is bounded."""
    assert form_of(q.F16, 64, 1, 32, 8, 128, 30720) == "parted" and form_of(q.F16, 16, 2, 24, 8, 64, 2240) == "16"
    assert form_of(q.I8, 64, 1, 32, 8, 128, 4000) == "16" and form_of(q.F16, 64, 1, 32, 8, 128, 4000) == "parted"
    assert form_of(q.I8, 64, 1, 32, 8, 128, 8000) == "parted"
    assert form_of(q.F16, 1024, 512, 8, 8, 64, 32) == "16" and form_of(q.F16, 1024, 512, 9, 9, 64, 32) == "whole"
    assert form_of(q.BF16, 1024, 512, 9, 9, 64, 2000) == "few"


def test_shared_as_many_tiles_as_slots():
    """16-column tiles of the prefixes, more than the slots they have: each has a workgroup, the longest are split."""
    shared(q.F16, 8, 8, 64, 16, [[(50, 3)] * 2 for _ in range(63)] + [[(2900, 5)] * 2], 15)
    shared(q.F8, 4, 4, 256, 16, [[(50, 3)] * 2 for _ in range(63)] + [[(2900, 5)] * 2], 16)
    shared(q.I8, 34, 1, 64, 16, [[(60, 1)] * 30 for _ in range(8)], 17)


def test_shared_behind_the_prefix_split_among_many():
    """As many sequences as slots, one of them long behind its prefix; and few of them, all split."""
    shared(q.F16, 8, 8, 64, 16, [[(30, 20)] * 65 + [(30, 3000)]], 12)
    shared(q.I8, 8, 8, 64, 16, [[(30, 20)] * 65 + [(30, 3000)]], 12)
    shared(q.F8, 16, 1, 64, 16, [[(1200, 3)] * 30 + [(1200, 2500)]], 13)


@pytest.mark.parametrize("kv_type", [q.F16, q.F8])
def test_shared_many_sequences_and_groups(kv_type):
    rng = np.random.default_rng(4)
    groups = [[(int(s), int(a)) for a in rng.integers(0, 40, m)]
              for s, m in zip(rng.integers(0, 150, 90), rng.integers(1, 5, 90))]
    shared(kv_type, 4, 2, 64, 16, groups, 5, outside=(3, 4))
    shared(kv_type, 4, 1, 64, 16, [[(200, int(a)) for a in rng.integers(0, 30, 600)]], 6)


@pytest.mark.parametrize("kv_type", ALL)
def test_shared_pages_of_the_others_are_not_read(kv_type):
    shared(kv_type, 6, 2, 64, 16, [[(100, 20), (100, 7), (48, 3)], [(300, 2), (300, 40)]], 7, bad_rest=True, gap=32)


@pytest.mark.parametrize("kv_type", ALL)
def test_shared_lengths_below_the_prefix(kv_type):
    """A padded slot, a length inside the prefix, one that ends with it; kv_len counts everywhere."""
    shared(kv_type, 4, 2, 128, 16, [[(150, 10), (150, 6), (150, 30), (150, 0), (150, 9)]], 8,
           lens=[160, 0, 70, 150, -3])


@pytest.mark.parametrize("kv_type", ALL)
def test_shared_promise_broken_and_bad_pages(kv_type):
    """A share larger than the first sequence's leaves positions out and sets the flag; so does a page of the
    prefix that is not there, for all its sequences."""
    nq, nkv, hd, page = 4, 1, 64, 16
    rng = np.random.default_rng(9)
    K, V = _draw(rng, [80, 100], nkv, hd)
    K[1][:64], V[1][:64] = K[0][:64], V[0][:64]
    c = Cache(kv_type, K, V, page, nkv, hd, rng)
    x = rng.standard_normal((2, nq * hd)).astype(np.float32)

    def run(share, keep):
        o = torch.full((2, nq * hd), float("nan"), device="cuda")
        ws = D.attn_workspace(q.OP_ATTN_SHARED, 2, nq, nkv, hd)
        q.qgemv_attn_shared(*c.args(), c.kv_len, 2, ints([0, 2]), ints(share), 1, dev(x), nq * hd, nq, 0.125, o, ws)
        parts = []
        for b in range(2):
            k, v = K[b][keep[b]], V[b][keep[b]]
            dv = scales64(v, kv_type) if kv_type in BYTES else np.ones(v.shape[:2])
            qr = x[b].reshape(nq, hd)
            parts.append(parts64(qr, held(k, kv_type), held(v, kv_type), dv, nkv, 0.125, len(k) - 1, kv_type))
        check_rows(host(o), parts, [80, 100], hd, kv_type, "left out")
        assert q.qgemv_attn_error(ws) == 1 and q.qgemv_attn_error(ws) == 0

    run([40, 64], [np.r_[0:80], np.r_[0:40, 64:100]])
    c.table[0, 1] = -1
    run([64, 64], [np.r_[0:16, 32:80], np.r_[0:16, 32:100]])


def test_shared_is_attention_without_groups():
    """The same batch by qgemv_attn, pages shared in its table: equal up to the tolerance of either."""
    c, x, o = shared(q.F16, 8, 2, 64, 16, [[(320, 20), (320, 50), (320, 1)]], 10)
    one = torch.empty((3, 8 * 64), device="cuda")
    ws = D.attn_workspace(q.OP_ATTN, 3, 8, 2, 64)
    q.qgemv_attn(*c.args(), c.kv_len, 3, dev(x), 12 * 64, 8, 64 ** -0.5, one, ws)
    assert np.abs(host(one) - o).max() <= 2e-5 * np.abs(o).max()


@pytest.mark.parametrize("kv_type", ALL)
@pytest.mark.parametrize("form,n,nq", [("16", 3, 4), ("parted", 130, 64)])
def test_shared_lengths_beyond_the_table(kv_type, form, n, nq):
    """Lengths and shares past the table's positions, a negative length and a negative share: what has no place is
    left out and flagged, and the workspace serves the next call."""
    nkv, hd, page, full = 1, 64, 16, 64
    assert form_of(kv_type, n, 1, nq, nkv, hd, full) == form
    rng = np.random.default_rng(21)
    K, V = _draw(rng, [full] * n, nkv, hd)
    for b in range(1, n):
        K[b], V[b] = K[0], V[0]
    c = Cache(kv_type, K, V, page, nkv, hd, rng, extra_entries=0)
    x = rng.standard_normal((n, nq * hd)).astype(np.float32)
    ws = D.attn_workspace(q.OP_ATTN_SHARED, n, nq, nkv, hd)
    hk, hv = held(K[0], kv_type), held(V[0], kv_type)
    dv = scales64(V[0], kv_type) if kv_type in BYTES else np.ones(V[0].shape[:2])

    def run(lens, share, flag):
        o = torch.full((n, nq * hd), float("nan"), device="cuda")
        q.qgemv_attn_shared(*c.args(), ints(lens), n, ints([0, n]), ints(share), 1, dev(x), nq * hd, nq, 0.125, o, ws)
        seen = [min(max(a, 0), full) for a in lens]
        parts = [parts64(x[b].reshape(nq, hd), hk, hv, dv, nkv, 0.125, seen[b] - 1, kv_type) for b in range(n)]
        check_rows(host(o), parts, seen, hd, kv_type, "beyond the table")
        assert q.qgemv_attn_error(ws) == flag

    run([2 ** 31 - 1, -5] + [40 + b % 30 for b in range(n - 2)], [2 ** 31 - 1] * n, 1)
    run([full] * n, [-2 ** 31] * n, 0)
    run([full] * n, [33] + [b % 34 for b in range(1, n)], 0)
